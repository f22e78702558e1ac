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
// workgroup of four waves makes a tile of 64 x 64, 32 of the reduction at a time
// through registers into LDS, element by element at ragged ends.  As in the tile
// kernels an operand stays as it lies in memory, and one whose reduction runs across
// the rows is read through the transposing load (turned at its store into LDS, element
// by element, the gradients below took 5.3 and 8.2 ms).  8 experts of 8191 x 4096,
// 16381 rows: 3.1 ms, gradients 2.9 and 2.6, a third of the tile kernels' rate: nothing
// is on its way while a tile is multiplied.
constexpr int kAnyTile = 64, kAnyDepth = 32;
constexpr int kAnyAlong = kAnyDepth + 8, kAnyAcross = kAnyTile + 8;  // a row's elements in LDS
constexpr int kAnyElements = kAnyTile * kAnyAlong;
static_assert(kAnyDepth * kAnyAcross <= kAnyElements, "either layout fits");

// An operand seen as [i, q], q along the reduction: one of its two strides is 1.
template <bool ALONG>  // q is the contiguous one
struct View {
  const uint16_t* base;
  int64_t ld;      // the other stride
  int n, depth;    // i < n, q < depth

  __device__ __forceinline__ void load(int i0, int q0, uint16_t* tile) const {
    const int u = threadIdx.x;
    const int r = ALONG ? u >> 2 : u >> 3, c = (ALONG ? u & 3 : u & 7) * 8;
    const int i = i0 + (ALONG ? r : c), q = q0 + (ALONG ? c : r);
    const bool in = i < n && q < depth;
    const uint16_t* p = base + (ALONG ? i * ld + q : q * ld + i);
    const int left = in ? (ALONG ? depth - q : n - i) : 0;
    dwords4 d{};
    if (left >= 8) {
      d = load16(p);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        d[j / 2] |= j < left ? static_cast<uint32_t>(p[j]) << (16 * (j & 1)) : 0u;
    }
    *reinterpret_cast<dwords4*>(tile + r * (ALONG ? kAnyAlong : kAnyAcross) + c) = d;
  }
  // The fragment of 16 i from `first` on: this lane's i and 8 q.
  static __device__ __forceinline__ dwords4 read(const uint16_t* tile, int first) {
    const int l = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    if constexpr (ALONG) {
      return *reinterpret_cast<const dwords4*>(tile + (first + l) * kAnyAlong + 8 * g);
    } else {
      typedef short v4i16 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) v4i16* LdsPtr;
      const uint16_t* p = tile + (8 * g + (l >> 2)) * kAnyAcross + first + (l & 3) * 4;
      const auto lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(p));
      const auto hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(p + 4 * kAnyAcross));
      const dwords2 a = __builtin_bit_cast(dwords2, lo), b = __builtin_bit_cast(dwords2, hi);
      return dwords4{a[0], a[1], b[0], b[1]};
    }
  }
};

template <Product P, typename T, typename TO>
__global__ __launch_bounds__(256) void grouped_any_kernel(GroupedArgs p, int col_tiles) {
  __shared__ __attribute__((aligned(16))) uint16_t xs[kAnyElements], ys[kAnyElements];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cols = P == Product::kOut ? p.N : p.K;
  int e, i0, i1, j0 = 0;
  View<P != Product::kWeights> x;
  View<P == Product::kOut> y;
  if constexpr (P == Product::kWeights) {
    const int at = blockIdx.x;
    e = blockIdx.y;
    i0 = at / col_tiles * kAnyTile;
    i1 = min(p.N, i0 + kAnyTile);
    j0 = at % col_tiles * kAnyTile;
    int r0, r1;
    segment(p, e, r0, r1);
    const int n = max(r1 - r0, 0);
    x = {p.x + r0 * p.x_ld, p.x_ld, p.N, n};
    y = {p.y + r0 * p.y_ld, p.y_ld, p.K, n};
  } else {
    const int mt = blockIdx.x / col_tiles;
    j0 = (blockIdx.x - mt * col_tiles) * kAnyTile;
    if (!find_tile(count_tiles(p.offsets, p.E, p.rows, kAnyTile), mt, e, i0, i1)) return;
    const uint16_t* w = p.y + static_cast<int64_t>(e) * p.N * p.K;
    const int depth = P == Product::kOut ? p.K : p.N;
    x = {p.x, p.x_ld, i1, depth};
    y = {w, p.K, cols, depth};
  }
  // wave w makes columns 16 w ... + 15 of all 64 rows
  const int col = lane & 15, g = lane >> 4;
  f32x4 acc[4] = {};
  for (int q = 0; q < x.depth; q += kAnyDepth) {
    x.load(i0, q, xs);
    y.load(j0, q, ys);
    __syncthreads();
    const dwords4 a = y.read(ys, wave * 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = mfma16(T{}, a, x.read(xs, i * 16), acc[i]);
    __syncthreads();
  }
  const int j = j0 + wave * 16 + 4 * g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i0 + i * 16 + col;
    if (row >= i1 || j >= cols) continue;
    if constexpr (P == Product::kWeights) {
      auto* o = static_cast<typename TO::bits*>(p.out) +
                (static_cast<int64_t>(e) * p.N + row) * p.K + j;
      f32x4 v = acc[i];
      if (p.accumulate) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (j + c < cols) v[c] += to_float(TO{}, o[c]);
      }
      store4<TO>(o, cols - j, v);
    } else {
      store4<TO>(static_cast<typename TO::bits*>(p.out) + row * p.out_ld + j, cols - j, acc[i]);
    }
  }
}

template <Product P>
void launch_any(const GroupedArgs& a, hipStream_t stream) {
  const int cols = P == Product::kOut ? a.N : a.K;
  const int col_tiles = (cols + kAnyTile - 1) / kAnyTile;
  const int64_t row_tiles = P == Product::kWeights ? (a.N + kAnyTile - 1) / kAnyTile
                                                   : a.rows / kAnyTile + (a.E < a.rows ? a.E : a.rows);
  // an expert's tiles along x, for which a launch's 2^32 threads are enough
  const dim3 grid(static_cast<unsigned>(row_tiles * col_tiles), P == Product::kWeights ? a.E : 1);
  with_types(a, [&](auto t, auto to) {
    hipLaunchKernelGGL((grouped_any_kernel<P, decltype(t), decltype(to)>), grid, dim3(256), 0,
                       stream, a, col_tiles);
  });
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
    case Product::kWeights:
      return tiles ? launch_grouped_weights(a, stream) : launch_any<Product::kWeights>(a, stream);
  }
}

}  // namespace moe
