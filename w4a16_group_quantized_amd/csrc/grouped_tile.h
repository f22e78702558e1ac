// The tile kernel of the grouped products (grouped_gemm.hip says what they are):
// C[i, j] = sum_q X[i, q] Y[j, q], output rows i, output columns j.
//
// A workgroup takes tiles of BM rows x BN columns, one after the other, and walks
// the reduction in chunks of 64, which go from memory straight to LDS in a ring of
// STAGES; the sequence of chunks runs on over the tiles.  An operand whose
// reduction is contiguous in memory is kept as rows of 128 bytes, their 16-byte
// blocks numbered xor a few bits of the row's, so that the 16-byte reads of 16
// rows meet all banks.  One whose reduction runs across the rows (W in the gradient
// of the rows, both operands in that of the weights) is kept as it lies, 64 rows of
// BM or BN values, and read through the transposing LDS load: 16 lanes fetch 4
// reduction rows x 16 values, and each gets the 4 of its own column.  There the
// blocks are numbered xor the row's two low bits, which sets the four rows of a
// read into different quarters of the banks.
//
// Fragments are read half a step (a step is 32 of the reduction; half of the wave's
// rows) ahead of their products, across the chunks too: the barrier that lets a chunk
// be replaced stands before the last half step's products, whose fragments are in
// registers by then, and behind it the next chunk's first fragments are read.  A wave
// so has products to issue on both sides of the one barrier of a chunk.
//
// 8192 cubed, 256 x 256 tiles, bf16: 780 us (1.41 PFLOP/s), its gradients 762 and 754.
// The matrix units are busy 70 % of the cycles there and the clock falls to 1.9 GHz of
// 2.4, so it is the power as much as the cycles that bounds it: the same loop took 9 %
// fewer cycles after its scalar steps were cut and 1 % less time; 32 x 32 matrix
// instructions, which move twice the sums, took 855 us; with all loads of a chunk hitting
// one chunk in L2 741.  Measured slower: the next chunk's loads all behind the barrier
// (weights 754 -> 815 us) or over three half steps (770), and three or four stages of
// smaller tiles.
// 512 experts of 1280 x 2560, 40960 rows, 128 x 128 tiles: 700 us (5.2 TB/s), gradient of
// the rows 770 (4.8): bound by reading the weights.  Gradient of the weights, 810 us (4.5
// TB/s): bound by writing it and by the two chunks of a tile, which add to the stores (with
// 10240 rows, one chunk, 590 us, 5.8 TB/s).  Waiting for a tile's stores later than at the
// next barrier gave nothing (840 -> 863 us).  Stores are nontemporal: with plain ones 878
// us against 840, and 569 against 385 at 2560 x 640.
#pragma once

#include "tiles.h"
#include "train.h"
#include "typed.h"

#include <type_traits>

namespace moe {

template <typename T>
struct Fragment;
template <>
struct Fragment<F16> {
  typedef _Float16 type __attribute__((ext_vector_type(8)));
};
template <>
struct Fragment<BF16> {
  typedef __bf16 type __attribute__((ext_vector_type(8)));
};

__device__ __forceinline__ f32x4 mfma16(F16, dwords4 a, dwords4 b, f32x4 c) {
  using V = Fragment<F16>::type;
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(V, a), __builtin_bit_cast(V, b),
                                                c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma16(BF16, dwords4 a, dwords4 b, f32x4 c) {
  using V = Fragment<BF16>::type;
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(V, a),
                                                 __builtin_bit_cast(V, b), c, 0, 0, 0);
}
// Rows [r0, r1) of expert e, inside the tensors whatever the offsets hold.  The offsets
// do not change while a kernel runs: loads through the scalar cache.
__device__ __forceinline__ void segment(const GroupedArgs& p, int e, int& r0, int& r1) {
  typedef const __attribute__((address_space(4))) int* Constants;
  const auto o = (Constants)(p.offsets);
  r0 = p.offsets == nullptr ? 0 : min(max(o[e], 0), p.rows);
  r1 = p.offsets == nullptr ? p.rows : min(max(o[e + 1], 0), p.rows);
}

constexpr int kGroupTiles = 4;
constexpr int kChunk = 64;      // of the reduction

// Part `n` of a segment: whole chunks to each part but the last.
__device__ __forceinline__ void part_of(const GroupedArgs& p, int n, int& r0, int& r1) {
  const int len = (p.by_parts(max(r1 - r0, 0) + p.parts - 1) + kChunk - 1) / kChunk * kChunk;
  const int64_t from = r0 + static_cast<int64_t>(n) * len;
  r0 = static_cast<int>(min(from, static_cast<int64_t>(r1)));
  r1 = min(r1, static_cast<int>(min(from + len, static_cast<int64_t>(INT32_MAX))));
}

constexpr int kChunkRow = 128;  // bytes of it in a row

// KS > 1 groups of WM x WN waves take KS chunks at once, one each, and add their sums in
// LDS at a tile's end, in a fixed order: few tiles of a long reduction then have KS times
// as many waves at work, and a barrier for KS chunks.
template <int BM_, int BN_, int WM_, int WN_, int STAGES_, int KS_ = 1>
struct GroupedShape {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, STAGES = STAGES_, KS = KS_;
  static constexpr int kGroup = WM * WN, kWaves = KS * kGroup;
  static constexpr int kDepth = KS * kChunk;                 // of the reduction per stage
  static constexpr int MT = BM / 16 / WM, NT = BN / 16 / WN;  // 16 x 16 results per wave
  static constexpr int kX = BM * kChunkRow, kY = BN * kChunkRow, kPart = kX + kY;
  static constexpr int kStage = KS * kPart;
  static constexpr int kLoadX = kX / 1024 / kGroup, kLoadY = kY / 1024 / kGroup;
  static constexpr int kLoads = kLoadX + kLoadY;              // per wave and stage
  static constexpr int kTurn = 128, kScratch = 16 * kTurn;    // results turn per wave, below
  static constexpr int kSums = KS / 2 * BM * BN * 4;          // of half of the groups
  static constexpr int per_cu(Product p) {
    return static_cast<int>(kGfx950LdsBytes) /
           (STAGES * kStage + kGroup * kScratch + kSums +
            (p == Product::kWeights ? 0 : static_cast<int>(sizeof(TileTable))));
  }
  static_assert(kLoadX * kGroup * 1024 == kX && kLoadY * kGroup * 1024 == kY, "loads divide evenly");
  static_assert(kLoads >= 2 && MT % 2 == 0, "chunks are requested and rows multiplied in halves");
  static_assert((KS & (KS - 1)) == 0, "sums are added in halves");
};

// One operand's way through memory: the range that begins with the next chunk (uniform),
// and this lane's offset in a chunk.  What changes from chunk to chunk is a few scalar
// steps: all waves take them between the same products.
template <int B, int WAVES, bool ALONG, int KS>
struct Stream {
  static constexpr int kLoad = B * kChunkRow / 1024 / WAVES;
  Descriptor range;
  uint32_t step, shrink;  // bytes to the next chunk, and what the range loses by it
  uint32_t lane_at, load_step, from;
  int depth_at;  // ALONG: where in the chunk this lane's values lie

  static __device__ __forceinline__ uint32_t swizzle(uint32_t row) {
    // the same for all of a lane's loads, WAVES * 8 rows apart
    if (ALONG) return WAVES > 1 ? (row >> 1) & 7 : row & 7;
    return B >= 128 ? ((row & 3) << 2) | ((row >> 2) & 2) : B == 64 ? (row & 3) << 1 : (row & 1) << 1;
  }
  // `part`: which of the stage's chunks this wave takes.
  __device__ __forceinline__ void init(int wave, int part, int64_t ld) {
    const uint32_t u = wave * 64 + (threadIdx.x & 63);
    constexpr uint32_t kBlocks = ALONG ? 8 : B / 8;  // of 16 bytes per row in LDS
    static_assert(ALONG || kBlocks >= 4, "the swizzle stays inside a row");
    const uint32_t row = u / kBlocks, blk = (u % kBlocks) ^ swizzle(row);
    const uint32_t chunk = ALONG ? kChunkRow : static_cast<uint32_t>(kChunk * ld * 2);
    lane_at = part * chunk + row * static_cast<uint32_t>(ld * 2) + blk * 16;
    load_step = WAVES * 64 / kBlocks * static_cast<uint32_t>(ld * 2);
    from = lane_at;
    depth_at = ALONG ? part * kChunk + blk * 8 : 0;
    step = KS * chunk;
  }
  // `bytes` (under 2^31) from `at` on hold the tile's rows; with fixed, of every chunk.
  __device__ __forceinline__ void aim(const uint16_t* at, int64_t bytes, bool fixed) {
    range = descriptor(at, static_cast<uint32_t>(bytes));
    shrink = fixed ? 0 : step;
  }
  // Nothing is fetched from here on.
  __device__ __forceinline__ void stop() { range.d[2] = shrink = step = 0; }
  // `depth` values of the reduction are left: blocks behind it become zeros, as rows
  // behind the range do.
  __device__ __forceinline__ void prepare(int depth) {
    if (ALONG) from = depth_at < depth ? lane_at : kOutOfRange;
  }
  // Part i of the chunk, into LDS from address `lds` on.
  __device__ __forceinline__ void load(uint32_t lds, int wave, int i) const {
    load16_to_lds(range, lds + (i * WAVES + wave) * 1024, from + i * load_step);
  }
  __device__ __forceinline__ void move_on() {
    const uint64_t at = (static_cast<uint64_t>(range.d[1]) << 32 | range.d[0]) + step;
    range.d[0] = static_cast<uint32_t>(at);
    range.d[1] = static_cast<uint32_t>(at >> 32);
    range.d[2] -= shrink;
  }
};

// What a lane reads of an operand: fragment i (16 rows or columns), step s (32 of the
// reduction) of the chunk at `st`.
template <int B, int WAVES, bool ALONG>
struct Reader {
  uint32_t base;
  __device__ __forceinline__ void init(int first) {  // the wave's first row or column
    const uint32_t l = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
    if constexpr (ALONG) {
      const uint32_t row = first + l;
      base = row * kChunkRow + (g ^ Stream<B, WAVES, true, 1>::swizzle(row)) * 16;
    } else {
      const uint32_t q = g * 8 + (l >> 2), c = first + (l & 3) * 4;
      const uint32_t blk = (c >> 3) ^ Stream<B, WAVES, false, 1>::swizzle(q);
      base = q * (B * 2) + blk * 16 + (c & 4) * 2;
    }
  }
  __device__ __forceinline__ dwords4 read(const uint8_t* st, int i, int s) const {
    if constexpr (ALONG) {
      return *reinterpret_cast<const dwords4*>(st + (base ^ (64 * s)) + i * 16 * kChunkRow);
    } else {
      typedef short v4i16 __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) v4i16* LdsPtr;
      const uint8_t* p = st + (base ^ (i * 32)) + s * 32 * B * 2;
      const auto lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(p));
      const auto hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((LdsPtr)(p + 4 * B * 2));
      const dwords2 a = __builtin_bit_cast(dwords2, lo), b = __builtin_bit_cast(dwords2, hi);
      return dwords4{a[0], a[1], b[0], b[1]};
    }
  }
};

template <typename S, Product P, typename T, typename TO>
__global__ __launch_bounds__(64 * S::kWaves) void grouped_tile_kernel(GroupedArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t ring[S::STAGES * S::kStage];
  __shared__ __attribute__((aligned(16))) uint8_t turn[S::kGroup * S::kScratch];
  __shared__ __attribute__((aligned(16))) uint8_t sums[S::kSums > 0 ? S::kSums : 16];
  __shared__ TileTable table;
  constexpr bool kAlongX = P != Product::kWeights, kAlongY = P == Product::kOut;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave / S::kGroup, in_group = wave % S::kGroup;
  const int wm = in_group / S::WN, wn = in_group % S::WN;
  const int cols = P == Product::kOut ? p.N : p.K;

  // Tiles in groups of kGroupTiles row tiles, rows fastest, and each XCD (the
  // workgroups of equal index mod 8) a contiguous run of them: the tiles that run
  // together share both operands in its L2.  Groups run across experts: 8 experts of 8192 x
  // 4096, 16381 rows, fetch 2.8 GB of 0.67 GB of operands.
  // The runs have as many tiles, not as much work, which in the gradient of the weights is the
  // expert's rows: with 64 of 512 experts, one run, holding 40137 of 40960 rows it takes 1925
  // us, evenly 810; with half of 16381 rows on one of 8, 2670 and 900.
  const int total = P == Product::kWeights
                        ? p.E * p.parts * p.row_tiles
                        : keep_tiles(count_tiles(p.offsets, p.E, p.rows, S::BM), table);
  const int all = total * p.col_tiles;
  const int run = (all + 7) >> 3;
  const int run0 = (blockIdx.x & 7) * run;
  const int run_n = min(run, all - run0);
  const int first_tile = blockIdx.x >> 3, step = gridDim.x >> 3;
  if (first_tile >= run_n) return;
  const int mine = (run_n - first_tile + step - 1) / step;
  struct Tile {
    int e, i0, i1, j0;  // rows [i0, i1) and columns from j0 on of the output (of block e)
    int r0, depth;      // kWeights: first row of the sums; how many terms they have
  };
  // Row and column tile of tile n of `rows` row tiles.
  auto place = [&](int n, int rows, int& row, int& column) {
    const int grp = p.by_group(n);
    const int in = n - grp * kGroupTiles * p.col_tiles;
    const int gm = min(kGroupTiles, rows - grp * kGroupTiles);
    column = gm == 4 ? in >> 2 : gm == 2 ? in >> 1 : gm == 1 ? in : __umulhi(in, 0x55555556u);
    row = grp * kGroupTiles + in - column * gm;
  };
  auto locate = [&](int j) {
    const int tile = run0 + first_tile + j * step;
    Tile t;
    int row, column;
    if constexpr (P == Product::kWeights) {
      t.e = p.by_expert(tile);
      place(tile - t.e * p.row_tiles * p.col_tiles, p.row_tiles, row, column);
      t.i0 = row * S::BM;
      t.i1 = min(p.N, t.i0 + S::BM);
      const int e = p.by_parts(t.e);
      int r1;
      segment(p, e, t.r0, r1);
      if (p.parts > 1) part_of(p, t.e - e * p.parts, t.r0, r1);
      t.depth = max(r1 - t.r0, 0);
    } else {
      place(tile, total, row, column);
      find_tile(kept_tiles(table, p.offsets, p.E, p.rows, S::BM, total), row, t.e, t.i0, t.i1);
      t.r0 = 0;
      t.depth = P == Product::kOut ? p.K : p.N;
    }
    t.j0 = column * S::BN;
    return t;
  };
  // an expert without rows still has a chunk (of zeros)
  auto chunks_of = [](const Tile& t) { return max(1, (t.depth + S::kDepth - 1) / S::kDepth); };

  // ---- loads: the tile and chunk that are requested next
  Stream<S::BM, S::kGroup, kAlongX, S::KS> sx;
  Stream<S::BN, S::kGroup, kAlongY, S::KS> sy;
  sx.init(in_group, part, p.x_ld);
  sy.init(in_group, part, P == Product::kWeights ? p.y_ld : p.K);
  int load_left = 0;  // of the reduction
  uint32_t tail_x = 0, tail_y = 0;  // kWeights: bytes from the last chunk to the rows' end
  auto aim = [&](const Tile& t) {
    load_left = t.depth;
    if constexpr (P == Product::kWeights) {
      // Rows of the segment, each from the tile's first column to the matrix's last.  What a
      // chunk's last row reads behind its end is the next chunk's, up to BM / 8 rows of it: the
      // range is open until two chunks are left.
      static_assert(S::BM / 8 <= S::kDepth && S::BN / 8 <= S::kDepth, "no further than a chunk");
      const int64_t n = (t.depth - 1) % S::kDepth;
      tail_x = t.depth > 0 ? static_cast<uint32_t>((n * p.x_ld + p.N - t.i0) * 2) : 0;
      tail_y = t.depth > 0 ? static_cast<uint32_t>((n * p.y_ld + p.K - t.j0) * 2) : 0;
      const bool open = t.depth > 2 * S::kDepth, two = t.depth > S::kDepth;
      sx.aim(p.x + t.r0 * p.x_ld + t.i0, open ? INT32_MAX : tail_x + (two ? sx.step : 0), true);
      sy.aim(p.y + t.r0 * p.y_ld + t.j0, open ? INT32_MAX : tail_y + (two ? sy.step : 0), true);
    } else {
      const int64_t w = static_cast<int64_t>(p.N) * p.K;
      const int64_t skip = P == Product::kOut ? static_cast<int64_t>(t.j0) * p.K : t.j0;
      sx.aim(p.x + t.i0 * p.x_ld, (static_cast<int64_t>(t.i1 - t.i0 - 1) * p.x_ld + t.depth) * 2,
             false);
      sy.aim(p.y + t.e * w + skip, (w - skip) * 2, false);
    }
  };
  // The tile that is requested now, and the one before it.  With two stages the tile that
  // is multiplied next is one of them: it need not be located again.
  int load_tile = 0;
  Tile ahead = locate(0), held = ahead;
  auto tile_of = [&](int n) {
    if constexpr (S::STAGES > 2) return locate(n);
    return load_tile == n ? ahead : held;
  };
  const uint32_t ring_at = lds_address(ring);
  uint32_t load_at = ring_at;
  // Half of the next chunk's loads are requested at a time; the second half moves on,
  // to the next tile behind a tile's last chunk.  Behind the last tile the loads have
  // empty ranges (nothing is fetched), so that the number on their way is the same.
  constexpr int kHalf = S::kLoads / 2;  // the first one, the smaller if they differ
  auto prepare = [&]() {
    sx.prepare(load_left);
    sy.prepare(load_left);
  };
  auto load = [&](int i) {
    if (i < S::kLoadX)
      sx.load(load_at + part * S::kPart, in_group, i);
    else
      sy.load(load_at + part * S::kPart + S::kX, in_group, i - S::kLoadX);
  };
  auto move_on = [&]() {
    load_left -= S::kDepth;
    load_at = load_at == ring_at + (S::STAGES - 1) * S::kStage ? ring_at : load_at + S::kStage;
    if (load_left > 0) {
      sx.move_on();
      sy.move_on();
      if (P == Product::kWeights && load_left <= 2 * S::kDepth) {
        const bool two = load_left > S::kDepth;
        sx.range.d[2] = tail_x + (two ? sx.step : 0);
        sy.range.d[2] = tail_y + (two ? sy.step : 0);
      }
    } else if (++load_tile < mine) {
      held = ahead;
      aim(ahead = locate(load_tile));
    } else {
      held = ahead;
      sx.stop();
      sy.stop();
      load_left = INT32_MAX;
      tail_x = tail_y = 0;
    }
  };

  // ---- products
  const int col = lane & 15, g = lane >> 4;
  Reader<S::BM, S::kGroup, kAlongX> rx;
  Reader<S::BN, S::kGroup, kAlongY> ry;
  rx.init(wm * S::MT * 16);
  ry.init(wn * S::NT * 16);
  f32x4 acc[S::NT][S::MT];
  constexpr int kRowsHalf = S::MT / 2;
  struct Rows {
    dwords4 f[kRowsHalf];
  };
  struct Columns {
    dwords4 f[S::NT];
  };
  auto read_rows = [&](const uint8_t* st, int s, int half) {
    Rows r;
#pragma unroll
    for (int i = 0; i < kRowsHalf; ++i) r.f[i] = rx.read(st, half * kRowsHalf + i, s);
    return r;
  };
  auto read_columns = [&](const uint8_t* st, int s) {
    Columns r;
#pragma unroll
    for (int j = 0; j < S::NT; ++j) r.f[j] = ry.read(st + S::kX, j, s);
    return r;
  };
  // Half of the wave's rows by all of its columns.  The reads in front of these products
  // stay in front of them: left alone, the compiler moves each next to its use, and the
  // matrix units wait for LDS.  REQUEST >= 0 requests that half of the next chunk between
  // the products: all of it behind the barrier at once keeps every wave from its products
  // until the loads are taken.
  auto multiply = [&](const Rows& x, const Columns& y, auto which, auto request, bool on) {
    constexpr int W = decltype(which)::value, REQUEST = decltype(request)::value;
    constexpr int kAll = kRowsHalf * S::NT;
    constexpr int kFrom = REQUEST == 1 ? kHalf : 0, kCount = REQUEST == 1 ? S::kLoads - kHalf : kHalf;
    __builtin_amdgcn_sched_barrier(0);
    if (on) {
#pragma unroll
      for (int i = 0; i < kRowsHalf; ++i)
#pragma unroll
        for (int j = 0; j < S::NT; ++j) {
          f32x4& c = acc[j][W * kRowsHalf + i];
          c = mfma16(T{}, y.f[j], x.f[i], c);
          const int n = i * S::NT + j;
          if constexpr (REQUEST >= 0) {
#pragma unroll
            for (int l = n * kCount / kAll; l < (n + 1) * kCount / kAll; ++l) {
              __builtin_amdgcn_sched_barrier(0);
              load(kFrom + l);
              __builtin_amdgcn_sched_barrier(0);
            }
          }
        }
    } else if constexpr (REQUEST >= 0) {
#pragma unroll
      for (int l = 0; l < kCount; ++l) load(kFrom + l);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // Whether half W of this wave's rows has any that is stored: the others' products are
  // left out, and so are those of a chunk's second step behind the reduction's end (8
  // experts of 8192 x 4096, 16381 rows: 1001 -> 975 us).  Not in the gradient of the
  // weights, whose tiles are whole but at the matrix's edge: 8192 cubed 769 us, with the
  // branches 798.
  auto has_rows = [&](const Tile& t, int W) {
    return P == Product::kWeights || t.i0 + (wm * S::MT + W * kRowsHalf) * 16 < t.i1;
  };
  constexpr std::integral_constant<int, -1> kNone{};
  constexpr std::integral_constant<int, 0> kFirst{};
  constexpr std::integral_constant<int, 1> kSecond{};

  // Zeros, or what the output holds, an element at a time and in front of the tile's products:
  // 8 experts of 8192 x 4096, 16381 rows, fp32 1040 -> 1405 us; 512 of 1280 x 2560, bf16, 810 ->
  // 3715.
  auto begin = [&](const Tile& t) {
#pragma unroll
    for (int j = 0; j < S::NT; ++j)
#pragma unroll
      for (int i = 0; i < S::MT; ++i) acc[j][i] = f32x4{};
    if constexpr (P == Product::kWeights) {
      if (!p.accumulate || t.depth == 0 || part > 0) return;
#pragma unroll
      for (int i = 0; i < S::MT; ++i) {
        const int row = t.i0 + (wm * S::MT + i) * 16 + col;
        const auto* o = static_cast<const typename TO::bits*>(p.out) +
                        (static_cast<int64_t>(t.e) * p.N + min(row, p.N - 1)) * p.K;
#pragma unroll
        for (int j = 0; j < S::NT; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int c = t.j0 + (wn * S::NT + j) * 16 + 4 * g + r;
            if (c < p.K) acc[j][i][r] = to_float(TO{}, o[c]);
          }
      }
    }
  };

  // acc[j][i][r] is column 16 j' + 4 g + r of row 16 i' + col.  Results turn in LDS, 16
  // rows x kTurn bytes of them at a time, so that eight neighbouring lanes store that many
  // contiguous bytes of a row.  `place` is this wave's; a row's 16-byte slots are stored
  // with their number xor a few bits of the row's.
  auto store = [&](const Tile& t, uint8_t* place, auto whole) {
    constexpr bool WHOLE = decltype(whole)::value;  // every row and column is there
    constexpr int kCols = S::kTurn / kBytes<TO>, kSlots = S::kTurn / 16, kRows = 64 / kSlots;
    constexpr int kWide = kCols < S::NT * 16 ? kCols : S::NT * 16;
    static_assert(S::NT * 16 % kWide == 0, "columns turn evenly");
    auto slot = [](int row, int n) { return (n ^ (row >> 1)) & (kSlots - 1); };
    // addresses are worked out here, not once for all tiles: they would hold registers
    // through the main loop
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int col = lane & 15, g = lane >> 4;
    const int64_t out_ld = P == Product::kWeights ? p.K : p.out_ld;
    auto* out = static_cast<typename TO::bits*>(p.out) +
                (P == Product::kWeights ? static_cast<int64_t>(t.e) * p.N * p.K : 0);
    // where this lane stores, from the first of 16 rows and kWide columns on
    const int in = lane % kSlots * (16 / kBytes<TO>);
    const int64_t lane_at = lane / kSlots * out_ld + in;
#pragma unroll
    for (int i = 0; i < S::MT; ++i) {
      const int row0 = t.i0 + (wm * S::MT + i) * 16;
      if (!WHOLE && row0 >= t.i1) break;
#pragma unroll
      for (int c0 = 0; c0 < S::NT * 16; c0 += kWide) {
#pragma unroll
        for (int c = 0; c < kWide; c += 16) {  // columns c0 + c + 4 g ... + 3
          const f32x4 v = acc[(c0 + c) / 16][i];
          const int at = (c + 4 * g) * kBytes<TO>;
          uint8_t* to = place + col * S::kTurn + slot(col, at >> 4) * 16;
          if constexpr (kBytes<TO> == 4)
            *reinterpret_cast<dwords4*>(to) = __builtin_bit_cast(dwords4, v);
          else
            *reinterpret_cast<dwords2*>(to + (at & 8)) = pack4<TO>(v);
        }
        asm volatile("" ::: "memory");  // other lanes read what this one wrote
        const int j0 = t.j0 + wn * S::NT * 16 + c0;
#pragma unroll
        for (int r = 0; r < 16; r += kRows) {
          const int row = r + lane / kSlots;
          const dwords4 d =
              *reinterpret_cast<const dwords4*>(place + row * S::kTurn + slot(row, lane) * 16);
          if (kWide < kCols && in >= kWide) continue;
          if (!WHOLE && row0 + row >= t.i1) continue;
          auto* o = out + ((row0 + r) * out_ld + j0) + lane_at;
          if (WHOLE || j0 + in + 16 / kBytes<TO> <= cols) {
            store16(o, d);
          } else {
#pragma unroll
            for (int x = 0; x < 16 / kBytes<TO>; ++x)
              if (j0 + in + x < cols)
                o[x] = static_cast<typename TO::bits>(
                    kBytes<TO> == 4 ? d[x % 4] : d[x / 2] >> (16 * (x & 1)));
          }
        }
        asm volatile("" ::: "memory");
      }
    }
  };
  // The groups' sums, added in halves until the first group holds them.
  auto join = [&]() {
#pragma unroll
    for (int h = S::KS / 2; h > 0; h >>= 1) {
      auto* at = reinterpret_cast<f32x4*>(sums) +
                 ((part % h) * S::kGroup + in_group) * S::MT * S::NT * 64 + lane;
      if (part >= h && part < 2 * h) {
#pragma unroll
        for (int j = 0; j < S::NT; ++j)
#pragma unroll
          for (int i = 0; i < S::MT; ++i) at[(j * S::MT + i) * 64] = acc[j][i];
      }
      wait_lds_and_barrier();
      if (part < h) {
#pragma unroll
        for (int j = 0; j < S::NT; ++j)
#pragma unroll
          for (int i = 0; i < S::MT; ++i) acc[j][i] += at[(j * S::MT + i) * 64];
      }
      wait_lds_and_barrier();
    }
  };

  aim(ahead);
#pragma unroll
  for (int s = 0; s < S::STAGES; ++s) {
    prepare();
#pragma unroll
    for (int i = 0; i < (s + 1 < S::STAGES ? S::kLoads : kHalf); ++i) load(i);
    if (s + 1 < S::STAGES) move_on();
  }
  wait_loads_and_barrier<(S::STAGES - 2) * S::kLoads + kHalf>();
  uint32_t stage = 0;
  Tile t = tile_of(0);
  int chunks = chunks_of(t);
  begin(t);
  Columns y = read_columns(ring + part * S::kPart, 0), y1;
  Rows x = read_rows(ring + part * S::kPart, 0, 0), x1;
  bool first = has_rows(t, 0), second = has_rows(t, 1);
  for (int n = 0, c = 0;;) {
    const bool more =
        P == Product::kWeights || t.depth - c * S::kDepth - part * kChunk > kChunk / 2;
    const uint8_t* st = ring + stage + part * S::kPart;
    x1 = read_rows(st, 0, 1);
    multiply(x, y, kFirst, kSecond, first);
    move_on();
    y1 = read_columns(st, 1);
    x = read_rows(st, 1, 0);
    multiply(x1, y, kSecond, kNone, second);
    x1 = read_rows(st, 1, 1);
    multiply(x, y1, kFirst, kNone, first && more);
    // every wave holds its last fragments of this chunk; the next one is there when
    // only those behind it are on their way (stores among them make the wait
    // longer, never too short)
    wait_loads_and_barrier<(S::STAGES - 2) * S::kLoads>();
    stage = stage + S::kStage == S::STAGES * S::kStage ? 0 : stage + S::kStage;
    prepare();
    y = read_columns(ring + stage + part * S::kPart, 0);
    x = read_rows(ring + stage + part * S::kPart, 0, 0);
    multiply(x1, y1, kSecond, kFirst, second && more);
    if (++c < chunks) continue;
    if constexpr (S::KS > 1) join();
    if (part > 0 || (P == Product::kWeights && p.accumulate && t.depth == 0)) {
      // nothing to store, or what is there stays
    } else if (t.i1 - t.i0 == S::BM && t.j0 + S::BN <= cols) {
      store(t, turn + in_group * S::kScratch, std::true_type{});
    } else {
      store(t, turn + in_group * S::kScratch, std::false_type{});
    }
    if (++n == mine) break;
    t = tile_of(n);
    chunks = chunks_of(t);
    c = 0;
    first = has_rows(t, 0);
    second = has_rows(t, 1);
    begin(t);
  }
  // no load into this workgroup's LDS outlives it
  __builtin_amdgcn_s_waitcnt(0x0F70);
}

// f(operand type, output type) for a product's dtype codes.
template <typename F>
void with_types(const GroupedArgs& a, F&& f) {
  with_dtype(a.out_dtype, [&](auto to) {
    if (a.dtype == MOE_F16)
      f(F16{}, to);
    else
      f(BF16{}, to);
  });
}

template <typename S, Product P>
void launch_grouped_tiles(const GroupedArgs& a, hipStream_t stream) {
  const int cols = P == Product::kOut ? a.N : a.K;
  GroupedArgs args = a;
  args.row_tiles = (a.N + S::BM - 1) / S::BM;
  args.col_tiles = (cols + S::BN - 1) / S::BN;
  args.by_expert = Divisor(args.row_tiles * args.col_tiles);
  args.by_group = Divisor(kGroupTiles * args.col_tiles);
  args.parts = a.parts > 1 ? a.parts : 1;
  args.by_parts = Divisor(args.parts);
  // at most one short tile per expert; no more workgroups than run at once
  const int64_t row_tiles =
      P == Product::kWeights ? static_cast<int64_t>(a.E) * args.parts * args.row_tiles
                             : a.rows / S::BM + (a.E < a.rows ? a.E : a.rows);
  const int64_t resident = static_cast<int64_t>(device_info().cus) * S::per_cu(P);
  static_assert(S::per_cu(P) >= 1, "the ring fits in LDS");
  const int64_t tiles = row_tiles * args.col_tiles, groups = tiles < resident ? tiles : resident;
  const dim3 grid(static_cast<unsigned>((groups + 7) / 8 * 8)), block(64 * S::kWaves);
  with_types(a, [&](auto t, auto to) {
    hipLaunchKernelGGL((grouped_tile_kernel<S, P, decltype(t), decltype(to)>), grid, block, 0,
                       stream, args);
  });
}

using Grouped256 = GroupedShape<256, 256, 2, 4, 2>;
using Grouped128 = GroupedShape<128, 128, 2, 2, 2>;
using Grouped64 = GroupedShape<64, 64, 2, 2, 4>;
using GroupedSplit = GroupedShape<32, 32, 1, 1, 2, 8>;

// What a product takes per chunk of the reduction with `tiles` tiles of a shape, in units of
// 10 ns: the time of a chunk where the tiles fill the compute units once, as often as they do.
//   256 x 256, one on a unit   1.5 us (8192 cubed: 512 chunks 790 us)
//   128 x 128, one             0.65 us (2048 cubed, 256 tiles, 32 chunks: 26 us)
//              two             1.0 us (2048 x 4096 x 4096, 512 tiles, 64 chunks: 64 us)
//   64 x 64,   one, two        0.37, 0.47 us (1000 x 1024 x 1024, 256 tiles, 16 chunks: 9.4 us;
//                              400 x 4096 x 4096, 448 tiles, 64 chunks: 31 us)
//              more            0.6 us a turn of two (2048 cubed, 1024 tiles: 33 us)
constexpr int64_t kUnits = 256;  // compute units of the chip that the rules go by
inline int64_t cost_of(int size, int64_t tiles) {
  const int64_t pairs = (tiles + 2 * kUnits - 1) / (2 * kUnits);
  if (size == 256) return 150 * ((tiles + kUnits - 1) / kUnits);
  if (size == 128) return tiles <= kUnits ? 65 : 100 * pairs;
  return tiles <= kUnits ? 37 : pairs <= 1 ? 47 : 60 * pairs;
}

// The tile's size of the least cost, of two equal ones the larger; tiles(size) counts.
template <typename F>
int pick_size(F&& tiles) {
  int best = 256;
  for (int size : {128, 64})
    if (cost_of(size, tiles(size)) < cost_of(best, tiles(best))) best = size;
  return best;
}

// Tiles of a product of rows: experts that hold `mean` rows each, more or less, so that their
// last tile is half full.
inline int64_t row_product_tiles(int64_t active, int64_t mean, int cols, int size) {
  const int64_t col_tiles = (cols + size - 1) / size;
  if (active == 1) return (mean + size - 1) / size * col_tiles;
  const int64_t all = active * col_tiles, tiles = all * (2 * mean + size) / (2 * size);
  return tiles > all ? tiles : all;
}

}  // namespace moe
