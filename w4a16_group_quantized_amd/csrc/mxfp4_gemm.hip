// Grouped product of MXFP4 rows with MXFP4 expert weights:
//   out[r, n] = sum_k A[r, k] W[e(r), n, k],   e(r): offsets[e] <= r < offsets[e + 1]
// on the scaled matrix instructions, which take E2M1 codes and E8M0 scales as
// they lie in memory: a lane's operand is one 16-byte block of 32 codes and
// one scale byte.  Products are exact, sums are fp32, and a result is rounded
// once, at its store.  Weights are the instruction's rows and tokens its
// columns, so a lane ends with consecutive n of one token.
//
// The gate/up form takes W13's gate and up rows of 32 columns of I together
// and ends with a = SiLU(gate) * up in fp32, which it stores as MXFP4 (the
// 32 columns are one block): the down product's operand, without a pass over
// fp32 rows in between.
#include "mxfp4.h"
#include "mxfp4_tile.h"
#include "typed.h"

#include <type_traits>

namespace moe {
namespace {

// ---------------------------------------------------------------- streaming --
// Few rows of few experts: bound by the latency of reading each active expert's
// weights once.  A wave takes 16 weight rows, straight from memory to registers
// in windows of 512 values of K (a row's 256 bytes of codes and 16 bytes of
// scales), two windows in flight; the up to 16 tokens of its tile come through
// the caches.  Four waves make a workgroup: 64 output columns, or the two halves
// of gate and up of 32 columns of I.
//
// SPLIT > 1 shares the windows of K out, to the four waves of a workgroup that
// then takes 16 columns, or to twice as many waves of a gate/up workgroup; their
// sums meet in LDS and are added in the order of the parts.  4096 x 4096, one row:
// 4.7 us (10.8 unsplit, 8.4 MB); 7168 x 7168, 9.4 us (17.6).  gate/up of 10 rows of
// 512 experts, 1280 x 2560: 8.8 us for 17 MB (9.6 unsplit, 11.8 with the tiles
// below, whose hundred workgroups leave half of the compute units idle).  Below
// four windows the split costs: 20 experts, 2048 x 1280: 8.6 us (7.6 unsplit).
// Gate/up in four shares is slower there (10.7) and 3 % faster for one long row.
// Three windows in flight or five waves per SIMD are slower.  (Weights in the
// memory-side cache throughout.)
constexpr int kTokens = 16;

struct Window {
  dwords4 w[4], a[4];
  dwords4 ws, as;
};

template <bool GATE_UP, typename TO, int SPLIT>
__global__ __launch_bounds__(GATE_UP ? 256 * SPLIT : 256) void mx_stream_kernel(MxGemmArgs p,
                                                                               int n_tiles) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mt = blockIdx.x / n_tiles, nt = blockIdx.x - mt * n_tiles;
  int e, r0, r1;
  if (!find_tile(count_tiles(p.offsets, p.E, p.rows, kTokens), mt, e, r0, r1)) return;

  const int blocks = p.K / 32;  // 32-value blocks per row
  const int sbytes = mx_scale_bytes(p.K);
  const int col = lane & 15, g = lane >> 4;
  const int I = p.N / 2;
  const int part = GATE_UP ? wave >> 2 : SPLIT > 1 ? wave : 0;  // of K
  const int n = GATE_UP ? ((wave >> 1) & 1) * I + nt * 32 + (wave & 1) * 16 + col
                        : (SPLIT > 1 ? nt * 16 : nt * 64 + wave * 16) + col;
  const bool n_ok = n < p.N;
  const auto rw = make_rsrc(p.w_codes + static_cast<int64_t>(e) * p.N * (p.K / 2),
                            static_cast<uint32_t>(p.N) * (p.K / 2));
  const auto rs = make_rsrc(p.w_scales + static_cast<int64_t>(e) * p.N * sbytes,
                            static_cast<uint32_t>(p.N) * sbytes);
  // out of range for every window: such a lane's loads return zero
  const uint32_t w_at = n_ok ? static_cast<uint32_t>(n) * (p.K / 2) : kOutOfRange;
  const uint32_t ws_at = n_ok ? static_cast<uint32_t>(n) * sbytes : kOutOfRange;
  const int row = r0 + col;
  const int64_t arow = row < r1 ? a_row(p, row) : -1;
  const uint8_t* ap = p.a_codes + (arow < 0 ? 0 : arow) * (p.K / 2);
  const uint8_t* sp = p.a_scales + (arow < 0 ? 0 : arow) * sbytes;

  // Lane group g takes block 4 i + g at step i, so a step reads 64 contiguous
  // bytes of each weight row.
  auto load = [&](Window& b, int win) {
    const int b0 = win * 16;
    if (b0 >= blocks) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int blk = b0 + 4 * i + g;
      b.w[i] = buffer_load16(rw, blk < blocks ? w_at + blk * 16 : kOutOfRange);
      b.a[i] = dwords4{};
      if (arow >= 0 && blk < blocks) b.a[i] = *reinterpret_cast<const dwords4*>(ap + blk * 16);
    }
    // scales by words of 4 blocks: a row's last window may hold fewer than 4
    b.ws = dwords4{};
    b.as = dwords4{};
    if (b0 + 12 < blocks) {
      b.ws = buffer_load16(rs, ws_at + b0);
      if (arow >= 0) b.as = load_words4(sp + b0);
    } else {
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (b0 + 4 * i < blocks) {
          b.ws[i] = buffer_load4(rs, ws_at + b0 + 4 * i);
          if (arow >= 0) b.as[i] = *reinterpret_cast<const uint32_t*>(sp + b0 + 4 * i);
        }
    }
  };
  f32x4 acc{};
  auto compute = [&](const Window& b, int win) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int blk = win * 16 + 4 * i;
      if (blk >= blocks) return;
      // this lane's scale byte to the word's low end; blocks behind K (their
      // codes are zero) get the scale 1, whatever the padding holds
      const bool in = blk + g < blocks;
      const uint32_t sw = in ? b.ws[i] >> (8 * g) : 127u;
      const uint32_t sa = in ? b.as[i] >> (8 * g) : 127u;
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(b.w[i]), operand(b.a[i]), acc,
                                                             kFp4, kFp4, 0, sw, 0, sa);
    }
  };
  const int windows = (blocks + 15) / 16;
  Window b0, b1;
  load(b0, part);
  load(b1, part + SPLIT);
  for (int w = part; w < windows; w += 2 * SPLIT) {
    compute(b0, w);
    load(b0, w + 2 * SPLIT);
    if (w + SPLIT < windows) compute(b1, w + SPLIT);
    load(b1, w + 3 * SPLIT);
  }

  // acc[i] is column n0 + 4 g + i of token r0 + col.  A row without a token is zeros
  // whatever the weights hold (its zeros times a NaN scale are NaN)
  if (arow < 0) acc = f32x4{};
  if constexpr (GATE_UP) {
    __shared__ float h[4 * SPLIT][16][17];
    gate_up_epilogue<SPLIT>(acc, h, wave, I, nt, r0, r1 - r0, p.act_codes, p.act_scales);
  } else if constexpr (SPLIT > 1) {
    __shared__ float h[4][16][17];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[wave][col][4 * g + i] = acc[i];
    __syncthreads();
    const int t = threadIdx.x >> 4, c = threadIdx.x & 15;
    if (r0 + t >= r1 || nt * 16 + c >= p.N) return;
    const float sum = ((h[0][t][c] + h[1][t][c]) + h[2][t][c]) + h[3][t][c];
    static_cast<typename TO::bits*>(p.out)[(r0 + t) * p.out_ld + nt * 16 + c] =
        from_float(TO{}, sum);
  } else {
    if (row >= r1) return;
    const int n0 = nt * 64 + wave * 16 + 4 * g;
    auto* o = static_cast<typename TO::bits*>(p.out) + row * p.out_ld + n0;
    store4<TO>(o, p.N - n0, acc);
  }
}

// ------------------------------------------------------------------- tiles --
// A workgroup takes tiles of BW weight rows x BT tokens, one after the other,
// and walks K in chunks of CB 32-value blocks (16 CB bytes of codes and CB of
// scales per row).  Chunks go from memory straight to LDS (no registers in
// between) in a ring of STAGES: the next one is requested as soon as its place
// is free, one barrier per chunk, and the sequence of chunks runs on over the
// tiles, so the loads of a tile are on their way while the one before is
// multiplied and stored.  In LDS a row's blocks are stored with their number
// xor a few bits of the row's, so that the 16-byte reads of 8 neighbouring rows
// meet different banks.
//
// 512 experts, 1280 x 2560: 217 us for 40960 rows (4.85 TB/s, bound by memory;
// one workgroup per tile, without the running ring, 252), 29 us for 80 rows
// (4.4 TB/s).  One expert, 8191 x 8192 x 8192: 282 to 301 us, 3.7 to 3.9
// PFLOP/s, 53 % of the cycles in matrix instructions at the clock it runs at.  Per
// chunk of 256 values a compute unit moves 192 KB of fragments out of LDS and 68 KB
// into it, about 2080 cycles at 128 bytes each, and its matrix instructions take
// 2048; a chunk takes about 4000, so the two hardly overlap: all eight waves start
// on fragment reads behind the chunk's one barrier.
//
// Tokens behind a segment and weight rows behind N leave what LDS holds, or
// rows that follow: each result depends on its own row and token only, and
// theirs are not stored.
template <int BW_, int BT_, int WW_, int WT_, int STAGES_>
struct TileShape {
  static constexpr int BW = BW_, BT = BT_, WW = WW_, WT = WT_, CB = 8, STAGES = STAGES_;
  static constexpr int kWaves = WW * WT;
  static constexpr int NW = BW / 32 / WW, NT = BT / 32 / WT;  // 32 x 32 results per wave
  static constexpr int kRow = 16 * CB;                        // bytes of codes per row and chunk
  static constexpr int kCodes = (BW + BT) * kRow;
  static constexpr int kStage = kCodes + (BW + BT) * CB;
  static constexpr int kRowsPerLoad = 1024 / kRow;            // a wave's load of 16 bytes per lane
  static constexpr int kLoadW = BW / kRowsPerLoad / kWaves, kLoadT = BT / kRowsPerLoad / kWaves;
  static constexpr int kSetRows = 256 / CB;                   // rows per load of scale words
  static constexpr int kSetsW = BW / kSetRows, kSetsT = (BT + kSetRows - 1) / kSetRows;
  static constexpr int kScaleW = (kSetsW + kWaves - 1) / kWaves;
  static constexpr int kScaleT = (kSetsT + kWaves - 1) / kWaves;
  static constexpr int kLoads = kLoadW + kLoadT + kScaleW + kScaleT;  // per wave and chunk
  static constexpr bool kTrim = BT == 32 && STAGES == 2;      // leave out blocks behind K
  static constexpr int kTurn = 128, kScratch = 32 * kTurn;    // results turn per wave, below
  static constexpr int kLds = STAGES * kStage + static_cast<int>(sizeof(TileTable));
  static constexpr int kPerCu = static_cast<int>(kGfx950LdsBytes) / kLds;
  static_assert(kLds <= static_cast<int>(kGfx950LdsBytes), "the ring fits in LDS");
  static_assert(kLoadW * kWaves * kRowsPerLoad == BW && kLoadT * kWaves * kRowsPerLoad == BT &&
                    kSetsW * kSetRows == BW && (BT % kSetRows == 0),
                "loads divide evenly");
  static_assert(kWaves * kScratch <= kStage, "results turn inside one stage");
};

template <typename S, bool GATE_UP, typename TO>
__global__ __launch_bounds__(64 * S::kWaves) void mx_tile_kernel(MxGemmArgs p, int n_tiles) {
  __shared__ __attribute__((aligned(16))) uint8_t ring[S::STAGES * S::kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ww = wave / S::WT, wt = wave % S::WT;

  // Tiles in groups of kGroupTiles token tiles, tokens fastest, and each XCD
  // (the workgroups of equal index mod 8) a contiguous run of them: the tiles
  // that run together share weight rows and tokens in its L2.
  constexpr int kGroupTiles = 4;
  __shared__ TileTable table;
  const int total = keep_tiles(count_tiles(p.offsets, p.E, p.rows, S::BT), table);
  const int all = total * n_tiles;
  const int run = (all + 7) >> 3;
  const int run0 = (blockIdx.x & 7) * run;
  const int run_n = min(run, all - run0);
  const int first_tile = blockIdx.x >> 3, step = gridDim.x >> 3;
  if (first_tile >= run_n) return;
  const int mine = (run_n - first_tile + step - 1) / step;
  struct Tile {
    int nt, e, r0, r1;
  };
  auto locate = [&](int j) {
    const int tile = run0 + first_tile + j * step;
    const int grp = tile / (kGroupTiles * n_tiles);
    const int in = tile - grp * kGroupTiles * n_tiles;
    const int gm = min(kGroupTiles, total - grp * kGroupTiles);
    Tile t{in / gm, 0, 0, 0};
    find_tile(kept_tiles(table, p.offsets, p.E, p.rows, S::BT, total),
              grp * kGroupTiles + in - t.nt * gm, t.e, t.r0, t.r1);
    return t;
  };

  const int blocks = p.K / 32, chunks = (blocks + S::CB - 1) / S::CB;
  const int row_bytes = p.K / 2, sbytes = mx_scale_bytes(p.K);
  const int I = p.N / 2;

  // ---- loads: the tile and chunk that are requested next
  Descriptor rw, rws, ra, ras;
  uint32_t at_w[S::kLoadW], at_t[S::kLoadT], at_ws[S::kScaleW], at_ts[S::kScaleT];
  auto swizzle = [](int row) { return (row >> 1) & 7; };
  // the set of rows whose scales this wave loads; spare waves repeat a load
  auto scale_set = [&](int i, int sets) { return (i * S::kWaves + wave) % sets; };
  auto aim = [&](const Tile& t) {
    rw = descriptor(p.w_codes + static_cast<int64_t>(t.e) * p.N * row_bytes,
                    static_cast<uint32_t>(p.N) * row_bytes);
    rws = descriptor(p.w_scales + static_cast<int64_t>(t.e) * p.N * sbytes,
                     static_cast<uint32_t>(p.N) * sbytes);
    const int64_t first = p.row_slots == nullptr ? t.r0 : 0;
    auto clip = [](int64_t n) { return static_cast<uint32_t>(n < INT32_MAX ? n : INT32_MAX); };
    ra = descriptor(p.a_codes + first * row_bytes, clip((p.a_rows - first) * row_bytes));
    ras = descriptor(p.a_scales + first * sbytes, clip((p.a_rows - first) * sbytes));
    // Weight row of tile row rr: gate/up alternates 32 gate and 32 up rows.
    auto w_row = [&](int rr) -> uint32_t {
      if constexpr (GATE_UP)
        return ((rr >> 5) & 1) * I + t.nt * (S::BW / 2) + (rr >> 6) * 32 + (rr & 31);
      else
        return t.nt * S::BW + rr;
    };
    // Offset of tile row tr's row of A in units of `bytes`; a row behind the
    // segment, or without a token, is not read.
    auto t_at = [&](int tr, int bytes) -> uint32_t {
      if (t.r0 + tr >= t.r1) return kOutOfRange;
      if (p.row_slots == nullptr) return static_cast<uint32_t>(tr) * bytes;
      const int64_t a = a_row(p, t.r0 + tr);
      return a < 0 ? kOutOfRange : static_cast<uint32_t>(a) * bytes;
    };
    const int in_row = lane / S::CB, at = lane % S::CB;  // this lane's part of a load
#pragma unroll
    for (int i = 0; i < S::kLoadW; ++i) {
      const int rr = (i * S::kWaves + wave) * S::kRowsPerLoad + in_row;
      at_w[i] = w_row(rr) * row_bytes + (at ^ swizzle(rr)) * 16;
    }
#pragma unroll
    for (int i = 0; i < S::kLoadT; ++i) {
      const int tr = (i * S::kWaves + wave) * S::kRowsPerLoad + in_row;
      at_t[i] = t_at(tr, row_bytes) + (at ^ swizzle(tr)) * 16;
    }
    const int set_row = lane / (S::CB / 4), word = lane % (S::CB / 4) * 4;
#pragma unroll
    for (int i = 0; i < S::kScaleW; ++i)
      at_ws[i] = w_row(scale_set(i, S::kSetsW) * S::kSetRows + set_row) * sbytes + word;
#pragma unroll
    for (int i = 0; i < S::kScaleT; ++i)
      at_ts[i] = t_at(scale_set(i, S::kSetsT) * S::kSetRows + set_row, sbytes) + word;
  };
  int load_tile = 0, load_chunk = 0;
  uint32_t load_at = lds_address(ring);
  const uint32_t ring_at = load_at;
  // Requests the next chunk.  Behind the last one the loads go to empty ranges
  // (nothing is fetched), so that the number on their way is always the same.
  auto load_next = [&]() {
    // Blocks of a last chunk that lie behind K belong to the next row.  The shape
    // for short K does not read them: at K = 640 they are a fifth of the weights'
    // bytes again (2560 rows of 512 experts 106 -> 104 us, 10240 rows 120 -> 117);
    // the test for it costs the others 1%.
    const int live = blocks - S::CB * load_chunk;
    auto behind = [&](int i) -> uint32_t {
      const int row = (i * S::kWaves + wave) * S::kRowsPerLoad + lane / S::CB;
      return (lane % S::CB ^ swizzle(row)) >= live ? kOutOfRange : 0u;
    };
    const bool whole = !S::kTrim || live >= S::CB;
#pragma unroll
    for (int i = 0; i < S::kLoadW; ++i) {
      load16_to_lds(rw, load_at + (i * S::kWaves + wave) * 1024,
                    whole ? at_w[i] : at_w[i] | behind(i));
      at_w[i] += S::kRow;
    }
#pragma unroll
    for (int i = 0; i < S::kLoadT; ++i) {
      load16_to_lds(ra, load_at + S::BW * S::kRow + (i * S::kWaves + wave) * 1024,
                    whole ? at_t[i] : at_t[i] | behind(i));
      at_t[i] += S::kRow;
    }
#pragma unroll
    for (int i = 0; i < S::kScaleW; ++i) {
      load4_to_lds(rws, load_at + S::kCodes + scale_set(i, S::kSetsW) * 256, at_ws[i]);
      at_ws[i] += S::CB;
    }
#pragma unroll
    for (int i = 0; i < S::kScaleT; ++i) {
      load4_to_lds(ras, load_at + S::kCodes + S::BW * S::CB + scale_set(i, S::kSetsT) * 256,
                   at_ts[i]);
      at_ts[i] += S::CB;
    }
    load_at = load_at == ring_at + (S::STAGES - 1) * S::kStage ? ring_at : load_at + S::kStage;
    ++load_chunk;
  };
  // Aims at the next tile when all of this one's chunks are requested.
  auto aim_next = [&]() {
    if (load_chunk < chunks) return;
    load_chunk = 0;
    if (++load_tile < mine)
      aim(locate(load_tile));
    else
      rw.d[2] = rws.d[2] = ra.d[2] = ras.d[2] = 0;
  };

  // ---- products
  const int col = lane & 31, g = lane >> 5;
  f32x16 acc[S::NW][S::NT];
  // Step s multiplies blocks 2s and 2s + 1 of the chunk, lane half g taking
  // block 2s + g; its scale byte is byte 2s + g of the row's.  The place of
  // block 2s + g is block g's xor 32 s; the fragments of one side differ by
  // whole 32 rows.
  const uint32_t in_rows = col * S::kRow + (g ^ swizzle(col)) * 16;
  const uint32_t at_wf = ww * S::NW * 32 * S::kRow + in_rows;
  const uint32_t at_tf = (S::BW + wt * S::NT * 32) * S::kRow + in_rows;
  const uint32_t at_w1 = S::kCodes + (ww * S::NW * 32 + col) * S::CB;
  const uint32_t at_t1 = S::kCodes + (S::BW + wt * S::NT * 32 + col) * S::CB;
  auto compute = [&](const uint8_t* st) {
    struct Step {
      dwords4 w[S::NW], t[S::NT];
    };
    struct alignas(S::CB) Scales {
      uint32_t v[S::CB / 4];
    };
    auto read = [&](int s) {
      Step f;
#pragma unroll
      for (int i = 0; i < S::NT; ++i)
        f.t[i] = *reinterpret_cast<const dwords4*>(st + (at_tf ^ (32 * s)) + i * 32 * S::kRow);
#pragma unroll
      for (int i = 0; i < S::NW; ++i)
        f.w[i] = *reinterpret_cast<const dwords4*>(st + (at_wf ^ (32 * s)) + i * 32 * S::kRow);
      return f;
    };
    auto scale = [&](uint32_t at, int i) {
      Scales v = *reinterpret_cast<const Scales*>(st + at + i * 32 * S::CB);
#pragma unroll
      for (int q = 0; q < S::CB / 4; ++q) v.v[q] >>= 8 * g;
      return v;
    };
    Scales ws[S::NW], ts[S::NT];
#pragma unroll
    for (int i = 0; i < S::NW; ++i) ws[i] = scale(at_w1, i);
#pragma unroll
    for (int i = 0; i < S::NT; ++i) ts[i] = scale(at_t1, i);
    auto multiply = [&](const Step& f, auto sc) {
      constexpr int s = decltype(sc)::value;
#pragma unroll
      for (int i = 0; i < S::NW; ++i)
#pragma unroll
        for (int j = 0; j < S::NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
              operand(f.w[i]), operand(f.t[j]), acc[i][j], kFp4, kFp4, 2 * (s & 1), ws[i].v[s / 2],
              2 * (s & 1), ts[j].v[s / 2]);
    };
    // the next step's reads go ahead of a step's products
    Step f0 = read(0), f1 = read(1);
    multiply(f0, std::integral_constant<int, 0>{});
    f0 = read(2);
    multiply(f1, std::integral_constant<int, 1>{});
    f1 = read(3);
    multiply(f0, std::integral_constant<int, 2>{});
    multiply(f1, std::integral_constant<int, 3>{});
  };
  // A last chunk of fewer blocks: the others become zeros of scale 1.
  auto cut = [&](uint8_t* st, int live) {
    for (int i = threadIdx.x; i < (S::BW + S::BT) * S::CB; i += 64 * S::kWaves) {
      const int row = i / S::CB, b = i % S::CB;
      if (b < live) continue;
      *reinterpret_cast<dwords4*>(st + row * S::kRow + (b ^ swizzle(row)) * 16) = dwords4{};
      st[S::kCodes + row * S::CB + b] = 127;
    }
  };

  // acc[i][j][4 q + r] is weight row 32 i' + 8 q + 4 g + r of token 32 j' + col.
  // Plain results turn in LDS, 32 tokens x kTurn bytes of them at a time, so
  // that eight neighbouring lanes store that many contiguous bytes of a token (straight from the registers a store's neighbouring lanes lie in
  // different rows, which took as long as half the products).  `turn` is this
  // wave's place; a token's 16-byte slots are stored with their number xor a few
  // bits of the token's.
  auto store = [&](const Tile& tl, uint8_t* turn) {
#pragma unroll
    for (int j = 0; j < S::NT; ++j) {
      const int row0 = tl.r0 + (wt * S::NT + j) * 32;
      const int row = row0 + col;
      if (row0 >= tl.r1) break;
      if constexpr (!GATE_UP) {
        const bool none = row < tl.r1 && p.row_slots != nullptr && a_row(p, row) < 0;
        constexpr int kCols = S::kTurn / kBytes<TO>, kSlots = S::kTurn / 16, kRows = 64 / kSlots;
        auto slot = [](int t, int n) { return (n ^ t) & (kSlots - 1); };
#pragma unroll
        for (int c0 = 0; c0 < S::NW * 32; c0 += kCols) {
#pragma unroll
          for (int e = 0; e < kCols; e += 8) {  // columns c0 + e + 4 g ... + 3
            f32x4 v;
#pragma unroll
            for (int r = 0; r < 4; ++r)
              v[r] = none ? 0.f : acc[(c0 + e) / 32][j][(c0 + e) % 32 / 2 + r];
            const int at = (e + 4 * g) * kBytes<TO>;
            uint8_t* to = turn + col * S::kTurn + slot(col, at >> 4) * 16;
            if constexpr (kBytes<TO> == 4)
              *reinterpret_cast<dwords4*>(to) = __builtin_bit_cast(dwords4, v);
            else
              *reinterpret_cast<dwords2*>(to + (at & 8)) = pack4<TO>(v);
          }
          const int n0 = tl.nt * S::BW + ww * S::NW * 32 + c0 + lane % kSlots * (16 / kBytes<TO>);
#pragma unroll
          for (int r = 0; r < 32; r += kRows) {
            const int t = r + lane / kSlots;
            const dwords4 d = *reinterpret_cast<const dwords4*>(turn + t * S::kTurn +
                                                                slot(t, lane) * 16);
            if (row0 + t >= tl.r1) continue;
            auto* o = static_cast<typename TO::bits*>(p.out) + (row0 + t) * p.out_ld + n0;
            if (n0 + 16 / kBytes<TO> <= p.N) {
              store16(o, d);
            } else {
#pragma unroll
              for (int x = 0; x < 16 / kBytes<TO>; ++x)
                if (n0 + x < p.N)
                  o[x] = static_cast<typename TO::bits>(
                      kBytes<TO> == 4 ? d[x % 4] : d[x / 2] >> (16 * (x & 1)));
            }
          }
        }
      } else {
        if (row >= tl.r1) continue;  // both lane halves of a token alike
        const bool none = p.row_slots != nullptr && a_row(p, row) < 0;
        const int sb = mx_scale_bytes(I);
#pragma unroll
        for (int i = 0; i < S::NW; i += 2) {
          const int blk = tl.nt * (S::BW / 64) + (ww * S::NW + i) / 2;
          float a[16];
          uint32_t m = 0;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            a[r] = none ? 0.f : silu_mul(acc[i][j][r], acc[i + 1][j][r]);
            m = max(m, abs_bits(a[r]));
          }
          m = max(m, static_cast<uint32_t>(__shfl_xor(m, 32, 64)));
          const uint32_t byte = mx_scale_byte(m);
          uint32_t h[4];  // four codes: half a word, whose other half the partner lane holds
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4)
            h[q4] = mx_pair(a[4 * q4], a[4 * q4 + 1], byte) |
                    (mx_pair(a[4 * q4 + 2], a[4 * q4 + 3], byte) << 8);
          // half 0 stores words 0 and 1, half 1 words 2 and 3
          const uint32_t give = g == 0 ? h[2] | (h[3] << 16) : h[0] | (h[1] << 16);
          const uint32_t got = __shfl_xor(give, 32, 64);
          uint2 w;
          w.x = g == 0 ? h[0] | (got << 16) : (got & 0xFFFFu) | (h[2] << 16);
          w.y = g == 0 ? h[1] | (got & 0xFFFF0000u) : (got >> 16) | (h[3] << 16);
          if (blk * 32 < I) {
            *reinterpret_cast<uint2*>(p.act_codes + static_cast<int64_t>(row) * (I / 2) +
                                      blk * 16 + g * 8) = w;
            if (g == 0)
              store_scale(p.act_scales + static_cast<int64_t>(row) * sb, blk, I / 32, sb, byte);
          }
        }
      }
    }
  };

  aim(locate(0));
#pragma unroll
  for (int s = 0; s + 1 < S::STAGES; ++s) {
    load_next();
    aim_next();
  }
  Tile now{};
  uint32_t stage = 0;
  for (int j = 0, c = 0;;) {
    // chunk c is there when only the chunks behind it are on their way (stores
    // among them make the wait longer, never too short)
    wait_loads_and_barrier<(S::STAGES - 2) * S::kLoads>();
    if (c == 0 && j > 0) {
      // through the stage that is free now
      const uint32_t free = stage == 0 ? (S::STAGES - 1) * S::kStage : stage - S::kStage;
      store(now, ring + free + wave * S::kScratch);
      if (j == mine) break;
      if constexpr (!GATE_UP) wait_lds_and_barrier();
    }
    load_next();
    aim_next();
    if (c == 0) {
      now = locate(j);
#pragma unroll
      for (int i = 0; i < S::NW; ++i)
#pragma unroll
        for (int t = 0; t < S::NT; ++t) acc[i][t] = f32x16{};
    }
    uint8_t* st = ring + stage;
    if (S::CB * (c + 1) > blocks) {
      cut(st, blocks - S::CB * c);
      wait_lds_and_barrier();
    }
    // a wave that multiplies goes before one that asks for loads (the dense
    // product of 8191 x 8192 x 8192: 290 -> 285 us)
    if constexpr (S::NW * S::NT >= 8) __builtin_amdgcn_s_setprio(1);
    compute(st);
    if constexpr (S::NW * S::NT >= 8) __builtin_amdgcn_s_setprio(0);
    stage = stage + S::kStage == S::STAGES * S::kStage ? 0 : stage + S::kStage;
    if (++c == chunks) {
      c = 0;
      ++j;
    }
  }
  // no load into this workgroup's LDS outlives it
  __builtin_amdgcn_s_waitcnt(0x0F70);
}

// Shapes, named by their tokens.  Those of 32 tokens take several workgroups per
// compute unit, two with a deep ring (K > 1024: 2560 rows of 512 experts, gate/up,
// 160 us against 164) or three with a short one (K = 640: 80 rows 19.4 against
// 22.9, 640 rows 80 against 88); the larger shapes fill LDS.
using Tile32 = TileShape<128, 32, 2, 1, 3>;
using Tile32Short = TileShape<128, 32, 2, 1, 2>;
using Tile64 = TileShape<256, 64, 4, 2, 3>;
using Tile128 = TileShape<256, 128, 4, 2, 3>;
using Tile256 = TileShape<256, 256, 4, 2, 2>;

template <typename S>
void launch_tiles(const MxGemmArgs& a, hipStream_t stream) {
  const bool gate_up = a.act_codes != nullptr;
  const int cols = gate_up ? S::BW / 2 : S::BW, width = gate_up ? a.N / 2 : a.N;
  const int n_tiles = (width + cols - 1) / cols;
  // at most one short tile per expert; no more workgroups than run at once
  const int64_t m_tiles = a.rows / S::BT + (a.E < a.rows ? a.E : a.rows);
  const int64_t resident = static_cast<int64_t>(device_info().cus) * S::kPerCu;
  const int64_t groups = m_tiles * n_tiles < resident ? m_tiles * n_tiles : resident;
  const dim3 grid(static_cast<unsigned>((groups + 7) / 8 * 8)), block(64 * S::kWaves);
  if constexpr (S::NW % 2 == 0) if (gate_up) {
    hipLaunchKernelGGL((mx_tile_kernel<S, true, F32>), grid, block, 0, stream, a, n_tiles);
    return;
  }
  with_dtype(a.out_dtype, [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL((mx_tile_kernel<S, false, T>), grid, block, 0, stream, a, n_tiles);
  });
}

template <bool GATE_UP, int SPLIT>
void launch_stream(const MxGemmArgs& a, hipStream_t stream) {
  const int cols = GATE_UP ? 32 : SPLIT > 1 ? 16 : 64;
  const int n_tiles = ((GATE_UP ? a.N / 2 : a.N) + cols - 1) / cols;
  // an expert's last tile may be partial: at most one more tile per expert
  const int m_tiles = a.rows / kTokens + (a.E < a.rows ? a.E : a.rows);
  const dim3 grid(static_cast<unsigned>(m_tiles) * n_tiles);
  if constexpr (GATE_UP) {
    hipLaunchKernelGGL((mx_stream_kernel<true, F32, SPLIT>), grid, dim3(256 * SPLIT), 0, stream, a,
                       n_tiles);
  } else {
    with_dtype(a.out_dtype, [&](auto t) {
      using T = decltype(t);
      hipLaunchKernelGGL((mx_stream_kernel<false, T, SPLIT>), grid, dim3(256), 0, stream, a, n_tiles);
    });
  }
}

void launch_stream(const MxGemmArgs& a, bool split, hipStream_t stream) {
  if (a.act_codes != nullptr)
    split ? launch_stream<true, 2>(a, stream) : launch_stream<true, 1>(a, stream);
  else
    split ? launch_stream<false, 4>(a, stream) : launch_stream<false, 1>(a, stream);
}

}  // namespace

// The rules go by the mean rows per expert; their figures are of rows shared out
// evenly.  Few experts that hold most of the rows take the shape that the mean gives.
void launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream) {
  const int active = a.E < a.rows ? a.E : a.rows;  // experts that can hold a row
  const int mean = a.rows / active;
  // the tile kernels address mapped rows of A with 31-bit offsets
  const bool far = a.row_slots != nullptr && a.a_rows * (a.K / 2) >= (static_cast<int64_t>(1) << 31);
  const int64_t weights = static_cast<int64_t>(active) * a.N * (a.K / 2);
  // gate/up of 512 experts, stream / tiles: 10 rows (17 MB) 8.8 / 11.8 us, 20 rows
  // (35 MB) 13.0 / 12.2, 80 rows 34.6 / 32.1, 2560 rows 216 / 160
  const bool light = mean <= 8 && weights <= 32 << 20;
  // products whose tiles would leave half of the compute units idle, stream /
  // tiles: 16384 x 16384, one row 30.5 / 48 us; 4096 x 4096, 48 rows 9.9 / 12.7;
  // 512 x 512 x K 2048 7.2 / 9.1; 32768 x 4096, 16 rows (256 tiles) 23.5 / 15.1;
  // gate/up 1280 x 2560, 40 rows 8.4 / 11.1; 4096 x 4096, 48 rows 12.7 / 13.5
  const int64_t tiles = static_cast<int64_t>(active) * ((mean + 15) / 16) * ((a.N + 127) / 128);
  const bool few = tiles <= 128;
  // the split needs a window for each of four waves
  if (far || light || few) return launch_stream(a, !far && a.K > 1536, stream);
  // the tile that holds the mean, or a smaller one where its tiles would leave
  // compute units without any (8192 x 8192 weights: 128 rows 46 us in 32 tiles of
  // 256 x 128, 21 in 256 of 128 x 32; 512 rows 63 and 39)
  const auto enough = [&](int bw, int bt) {
    return static_cast<int64_t>(active) * ((mean + bt - 1) / bt) * ((a.N + bw - 1) / bw) >=
           device_info().cus;
  };
  if (mean >= 512 && enough(256, 256)) return launch_tiles<Tile256>(a, stream);
  if (mean > 48 && enough(256, 128)) return launch_tiles<Tile128>(a, stream);
  if (mean > 24 && enough(256, 64)) return launch_tiles<Tile64>(a, stream);
  if (a.K > 1024) return launch_tiles<Tile32>(a, stream);
  launch_tiles<Tile32Short>(a, stream);
}

}  // namespace moe
