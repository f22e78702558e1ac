// Products of rows with their expert's weights, and their gradients, in fp16 and
// bf16 on the matrix instructions:
//   out[r, n]       = sum_k a[r, k] W[e, n, k]         offsets[e] <= r < offsets[e + 1]
//   grad_a[r, k]    = sum_n grad[r, n] W[e, n, k]
//   grad_w[e, n, k] = sum_r grad[r, n] a[r, k]         over the rows r of expert e
// Products are exact, sums are fp32 in a fixed order, and a result is rounded
// once, at its store.  The operand that runs along the output's columns is the
// instruction's rows, so a lane ends with consecutive columns of one output row.
#include "grouped_tile.h"

namespace moe {
namespace {

// ------------------------------------------------------------- any alignment --
// Sizes, strides and addresses that the tile kernels' 16-byte loads do not take: a
// workgroup of four waves makes a tile of 128 x 128 (64 x 64 where those are few), 64 of
// the reduction at a time (32 of the weights' gradient, whose operands both lie in long
// rows: 1640 us against 1755) through registers into one of two LDS buffers, so that the
// next ones are on their way while these are multiplied.  Loads are 16 bytes at any
// address; at a row's end they are the row's last 16 bytes, moved down on their way to LDS
// (element by element: 1675 -> 2133 us for one column less).  As in the tile kernels an
// operand stays as it lies in memory, and one whose reduction runs across the rows is read
// through the transposing load.  8192 x 8192 x 8190: 1500 us, gradients 1450 and 1350; 8
// experts of 8191 x 4096, 16381 rows: 1760, 1690 and 1450 (with one buffer and tiles of 64
// x 64 3090, 2930 and 2590): half of the tile kernels' rate.  What bounds it is the way
// through registers; loads that straddle cache lines come on top where an operand's rows are
// off the grid (all of 8192 x 8192 x 8190; the gradients' rows of 8191), which those of the
// product of 8191 x 4096 are not: N alone is odd there, and only its stores see it.
// 8 values without the first n, zeros behind the rest.
__device__ __forceinline__ dwords4 moved_down(dwords4 d, int n) {
  uint64_t lo = d[0] | static_cast<uint64_t>(d[1]) << 32, hi = d[2] | static_cast<uint64_t>(d[3]) << 32;
  if (n >= 4) {
    lo = n < 8 ? hi >> (16 * (n - 4)) : 0;
    hi = 0;
  } else if (n > 0) {
    lo = lo >> (16 * n) | hi << (64 - 16 * n);
    hi >>= 16 * n;
  }
  return dwords4{static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                 static_cast<uint32_t>(hi >> 32)};
}

// An operand seen as [i, q], q along the reduction: one of its two strides is 1.
template <bool ALONG, int TILE, int DEPTH>  // ALONG: q is the contiguous one
struct View {
  static constexpr int kRowBlocks = ALONG ? DEPTH / 8 : TILE / 8;  // of 8 in a row
  static constexpr int kRows = 256 / kRowBlocks, kLoads = (ALONG ? TILE : DEPTH) / kRows;
  static constexpr int kRow = (ALONG ? DEPTH : TILE) + 8;          // a row in LDS
  static constexpr int kElements = (ALONG ? TILE : DEPTH) * kRow;
  static_assert(kLoads >= 1, "every thread loads");
  const uint16_t* at;  // this thread's first 8 values of the chunk
  int64_t rows_ld, step;
  int i, q, n, depth;  // where they are; i < n, q < depth are there
  int lack;            // values that the chunk's 8 have less than 8
  dwords4 d[kLoads];

  __device__ __forceinline__ void init(const uint16_t* base, int64_t ld, int i0, int n_, int depth_) {
    const int r = threadIdx.x / kRowBlocks, c = threadIdx.x % kRowBlocks * 8;
    i = i0 + (ALONG ? r : c);
    q = ALONG ? c : r;
    n = n_;
    depth = depth_;
    at = base + (ALONG ? i * ld + q : q * ld + i);
    rows_ld = kRows * ld;
    step = ALONG ? DEPTH : DEPTH * ld;
  }
  // The next chunk, on its way into registers.  At a ragged end the last 8 values of the
  // row are loaded and moved down when they are put: to look at them here would wait.
  __device__ __forceinline__ void fetch() {
    const int size = ALONG ? depth : n, from = ALONG ? q : i;
    lack = size >= 8 ? max(0, from + 8 - size) : 0;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int ik = ALONG ? i + k * kRows : i, qk = ALONG ? q : q + k * kRows;
      d[k] = dwords4{};
      if (ik >= n || qk >= depth) continue;
      const uint16_t* p = at + k * rows_ld;
      if (size >= 8) {
        d[k] = load16(p - lack);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          d[k][j / 2] |= from + j < size ? static_cast<uint32_t>(p[j]) << (16 * (j & 1)) : 0u;
      }
    }
    at += step;
    q += DEPTH;
  }
  __device__ __forceinline__ void put(uint16_t* tile) {
    const int r = threadIdx.x / kRowBlocks, c = threadIdx.x % kRowBlocks * 8;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      if (lack > 0) d[k] = moved_down(d[k], lack);
      *reinterpret_cast<dwords4*>(tile + (r + k * kRows) * kRow + c) = d[k];
    }
  }
  // The fragment of 16 i from `first` on, step s (32 of the reduction): this lane's i and
  // 8 q.
  static __device__ __forceinline__ dwords4 read(const uint16_t* tile, int first, int s) {
    const int l = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    if constexpr (ALONG) {
      return *reinterpret_cast<const dwords4*>(tile + (first + l) * kRow + 32 * s + 8 * g);
    } else {
      typedef short v4i16 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) v4i16* LdsPtr;
      const uint16_t* p = tile + (32 * s + 8 * g + (l >> 2)) * kRow + first + (l & 3) * 4;
      const auto lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(p));
      const auto hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(p + 4 * kRow));
      const dwords2 a = __builtin_bit_cast(dwords2, lo), b = __builtin_bit_cast(dwords2, hi);
      return dwords4{a[0], a[1], b[0], b[1]};
    }
  }
};

template <int TILE, Product P, typename T, typename TO>
__global__ __launch_bounds__(256) void grouped_any_kernel(GroupedArgs p) {
  constexpr int DEPTH = P == Product::kWeights ? 32 : 64;
  using X = View<P != Product::kWeights, TILE, DEPTH>;
  using Y = View<P == Product::kOut, TILE, DEPTH>;
  __shared__ __attribute__((aligned(16))) uint16_t xs[2][X::kElements], ys[2][Y::kElements];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cols = P == Product::kOut ? p.N : p.K;
  // tiles in groups of kGroupTiles row tiles, each XCD a contiguous run, as in the tile
  // kernels; those behind the last have nothing to do
  const int tile = (blockIdx.x & 7) * (gridDim.x >> 3) + (blockIdx.x >> 3);
  const int grp = p.by_group(tile), in = tile - grp * kGroupTiles * p.col_tiles;
  const int mt = grp * kGroupTiles + in % kGroupTiles, j0 = in / kGroupTiles * TILE;
  int e, i0, i1;
  X x;
  Y y;
  int depth;
  if constexpr (P == Product::kWeights) {
    if (mt >= p.row_tiles) return;
    e = blockIdx.y;
    i0 = mt * TILE;
    i1 = min(p.N, i0 + TILE);
    int r0, r1;
    segment(p, e, r0, r1);
    if (p.parts > 1) part_of(p, blockIdx.z, r0, r1);
    e = e * p.parts + blockIdx.z;
    depth = max(r1 - r0, 0);
    x.init(p.x + r0 * p.x_ld, p.x_ld, i0, p.N, depth);
    y.init(p.y + r0 * p.y_ld, p.y_ld, j0, p.K, depth);
  } else {
    if (!find_tile(count_tiles(p.offsets, p.E, p.rows, TILE), mt, e, i0, i1)) return;
    depth = P == Product::kOut ? p.K : p.N;
    x.init(p.x, p.x_ld, i0, i1, depth);
    y.init(p.y + static_cast<int64_t>(e) * p.N * p.K, p.K, j0, cols, depth);
  }
  // each wave makes a quarter of the tile
  constexpr int F = TILE / 32;
  const int wm = (wave >> 1) * (TILE / 2), wn = (wave & 1) * (TILE / 2);
  const int col = lane & 15, g = lane >> 4;
  f32x4 acc[F][F] = {};
  x.fetch();
  y.fetch();
  for (int q = 0, b = 0; q < depth; q += DEPTH, b ^= 1) {
    x.put(xs[b]);
    y.put(ys[b]);
    __syncthreads();  // and every wave has read what the next chunk replaces
    x.fetch();
    y.fetch();
#pragma unroll
    for (int s = 0; s < DEPTH / 32; ++s) {
      dwords4 xf[F], yf[F];
#pragma unroll
      for (int i = 0; i < F; ++i) xf[i] = X::read(xs[b], wm + i * 16, s);
#pragma unroll
      for (int j = 0; j < F; ++j) yf[j] = Y::read(ys[b], wn + j * 16, s);
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) acc[i][j] = mfma16(T{}, yf[j], xf[i], acc[i][j]);
    }
  }
  // results turn in LDS, 16 rows of a wave's columns at a time, and are stored 8 to a lane
  constexpr int kWide = TILE / 2, kTurn = kWide + 4, kLanes = kWide / 8;
  static_assert(sizeof(xs) >= 4 * 16 * kTurn * sizeof(float), "the results turn in an operand's LDS");
  __syncthreads();
  float* turn = reinterpret_cast<float*>(xs) + wave * 16 * kTurn;
  const int c = j0 + wn + lane % kLanes * 8;
#pragma unroll
  for (int i = 0; i < F; ++i) {
#pragma unroll
    for (int j = 0; j < F; ++j)
      *reinterpret_cast<f32x4*>(turn + col * kTurn + j * 16 + 4 * g) = acc[i][j];
    asm volatile("" ::: "memory");  // other lanes read what this one wrote
#pragma unroll
    for (int r = lane / kLanes; r < 16; r += 64 / kLanes) {
      float v[8], held[8] = {};
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = turn[r * kTurn + lane % kLanes * 8 + k];
      const int row = i0 + wm + i * 16 + r;
      if (row >= i1 || c >= cols) continue;
      auto* o = static_cast<typename TO::bits*>(p.out) + c +
                (P == Product::kWeights ? (static_cast<int64_t>(e) * p.N + row) * p.K : row * p.out_ld);
      if (P == Product::kWeights && p.accumulate) {
        load8<TO>(o, cols - c, held);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += held[k];
      }
      // rows end inside a cache line, whose rest another lane stores: not nontemporal (weights
      // of 512 experts of 1280 x 2559, 80 rows: 2068 -> 1097 us)
      store8<TO, false>(o, cols - c, v);
    }
    asm volatile("" ::: "memory");
  }
}

template <int TILE, Product P>
void launch_any_tiles(const GroupedArgs& a, hipStream_t stream) {
  const int cols = P == Product::kOut ? a.N : a.K;
  GroupedArgs args = a;
  args.col_tiles = (cols + TILE - 1) / TILE;
  args.row_tiles = P == Product::kWeights ? (a.N + TILE - 1) / TILE
                                          : a.rows / TILE + (a.E < a.rows ? a.E : a.rows);
  args.by_group = Divisor(kGroupTiles * args.col_tiles);
  // whole groups, in eight runs; of an expert's tiles, which a launch's 2^32 threads take
  const int64_t rows = (args.row_tiles + kGroupTiles - 1) / kGroupTiles * kGroupTiles;
  const int64_t tiles = (rows * args.col_tiles + 7) / 8 * 8;
  const bool weights = P == Product::kWeights;
  const dim3 grid(static_cast<unsigned>(tiles), weights ? a.E : 1, weights ? a.parts : 1);
  with_types(a, [&](auto t, auto to) {
    hipLaunchKernelGGL((grouped_any_kernel<TILE, P, decltype(t), decltype(to)>), grid, dim3(256), 0,
                       stream, args);
  });
}

// Tiles of 128 x 128 where there is one for each compute unit and most of it is rows (2048
// x 2047 x 1023, 256 tiles: 33 us, with tiles of 64 x 64 39; 1000 x 1000 x 1023, 64: 24 and
// 15; 64 experts of 511 x 1023, 2000 rows, 256: 29 and 21).
template <Product P>
void launch_any(const GroupedArgs& a, hipStream_t stream) {
  const int cols = P == Product::kOut ? a.N : a.K;
  const int64_t active = a.E < a.rows ? a.E : a.rows, mean = active > 0 ? a.rows / active : 0;
  const int64_t col_tiles = (cols + 127) / 128;
  const int64_t row_tiles = P == Product::kWeights ? static_cast<int64_t>(a.E) * a.parts * ((a.N + 127) / 128)
                                                   : active * ((mean + 127) / 128);
  if (mean >= 64 && row_tiles * col_tiles >= kUnits)
    launch_any_tiles<128, P>(a, stream);
  else
    launch_any_tiles<64, P>(a, stream);
}

}  // namespace

// What the tile kernels' 16-byte loads and 32-bit offsets take.
static bool tiles_take(Product p, const GroupedArgs& a) {
  auto whole = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
  constexpr int64_t kMaxLd = 1 << 20;
  if (a.N % 8 || a.K % 8 || a.x_ld % 8 || a.x_ld > kMaxLd || !whole(a.x) || !whole(a.y)) return false;
  return p != Product::kWeights || (a.y_ld % 8 == 0 && a.y_ld <= kMaxLd);
}

void launch_grouped(Product p, const GroupedArgs& a, hipStream_t stream) {
  const bool tiles = tiles_take(p, a);
  switch (p) {
    case Product::kOut: return tiles ? launch_grouped_out(a, stream) : launch_any<Product::kOut>(a, stream);
    case Product::kRows: return tiles ? launch_grouped_rows(a, stream) : launch_any<Product::kRows>(a, stream);
    case Product::kWeights: {
      if (tiles) return launch_grouped_weights(a, stream);
      const GroupedArgs b = grouped_part_sums(a);
      launch_any<Product::kWeights>(b, stream);
      return launch_add_parts(a, b.parts, stream);
    }
  }
}

}  // namespace moe
