// The MXFP4 layer for one to six tokens in two launches.
//
// With so few tokens the five launches of the layer's steps (router and
// permutation, quantisation, gate/up, down, combine) are latency: 33.6 us at one
// token of 512 experts, 10 chosen, hidden 2560, intermediate 640, for 26 MB of
// weights; 17.4 us in these two (24 against 44 at two tokens, 41 against 60 at
// four, 52 against 63 at five, 64 against 73 at six).  Those are of four sets of
// inputs in turn, whose weights stay in the memory-side cache up to two tokens; from
// HBM one token takes 19.6 and two 26.2.  Here every workgroup does the small steps
// for itself:
//   gate/up  routes the tokens (one wave each) while its other waves quantise
//            them into LDS, then takes 32 columns of I of one expert, as the
//            streaming product does
//   down     takes 16 columns of H of every active expert, an expert per wave,
//            meets their rows in LDS and adds them up with the router's weights
// The sums' order is fixed: K's shares of gate/up in turn, down from k = 0 up.
#include "mxfp4_tile.h"
#include "route.h"

namespace moe {
namespace {

constexpr int kMaxSlots = 64;  // one slot per lane
constexpr int kMaxTokens = kMxSmallTokens;

// The permutation of at most 64 slots, lane s holding slot s (id < 0: none):
// the slot's row (slots ascending by expert, then by slot), and the ordinal of
// its expert among those that hold a slot.
struct Places {
  int row, ordinal;
};
__device__ __forceinline__ Places place_slots(int id, int S) {
  const int lane = threadIdx.x & 63;
  // distinct keys below 2^31: experts are fewer than 2^24
  const int key = lane < S ? id * 64 + lane : INT32_MAX;
  int row = 0;
  for (int q = 0; q < S; ++q) row += __builtin_amdgcn_readlane(key, q) < key;
  // the ids in the order of rows: an expert starts where they change
  const int sorted = __builtin_amdgcn_ds_permute(row * 4, id);
  const int before = __shfl_up(sorted, 1);  // in all lanes, the comparison's branch behind it
  const unsigned long long firsts = __ballot(lane < S && (lane == 0 || sorted != before));
  const int ordinal = __popcll(firsts & ((2ull << row) - 1)) - 1;
  return {row, ordinal};
}

// The lanes of the n-th active expert's slots (0: there is none).
__device__ __forceinline__ unsigned long long slots_of(const Places& p, int S, int n) {
  return __ballot((threadIdx.x & 63) < static_cast<unsigned>(S) && p.ordinal == n);
}

// Top-k of one token's E logits by one wave, as wave_topk gives it, for a short
// list: the top_k-th largest of the lanes' maxima is a bound that all of the
// top_k largest logits reach, few others do, and the reaching ones, one per
// lane, are ranked by counting.  A token with more than 64 of them (ties) goes
// to wave_topk.  0.6 us less than its top_k dependent rounds at top_k = 10.
template <int NPL>
__device__ __forceinline__ void small_topk(const float* __restrict__ row, int E, int top_k,
                                           uint64_t* list, int& my_id, float& my_logit,
                                           float& top_logit) {
  const int lane = threadIdx.x & 63;
  uint64_t key[NPL], best = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = lane + 64 * i;
    key[i] = e < E ? logit_key(row[e], e) : 0ull;
    best = max64(best, key[i]);
  }
  // the rank of this lane's maximum among the lanes' (keys are distinct; lanes
  // without an expert hold 0 and tie, behind all others)
  const uint32_t hi = static_cast<uint32_t>(best >> 32), lo = static_cast<uint32_t>(best);
  int rank = 0;
#pragma unroll
  for (int q = 0; q < 64; ++q) {
    const uint64_t other = (static_cast<uint64_t>(__builtin_amdgcn_readlane(hi, q)) << 32) |
                           static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, q));
    rank += other > best;
  }
  const unsigned long long bound_lane = __ballot(rank == min(top_k, min(E, 64)) - 1);
  uint64_t bound = 0;
  if (top_k <= 64 && bound_lane) {
    const int q = __builtin_ctzll(bound_lane);
    bound = (static_cast<uint64_t>(__builtin_amdgcn_readlane(hi, q)) << 32) |
            static_cast<uint32_t>(__builtin_amdgcn_readlane(lo, q));
  }
  int found = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const bool in = key[i] != 0 && key[i] >= bound;
    const unsigned long long who = __ballot(in);
    const int at = found + __popcll(who & ((1ull << lane) - 1ull));
    if (in && at < 64) list[at] = key[i];
    found += __popcll(who);
  }
  if (found > 64) return wave_topk<NPL>(row, E, top_k, my_id, my_logit, top_logit);
  const uint64_t mine = lane < found ? list[lane] : 0;
  int place = 0;
  for (int q = 0; q < found; ++q) place += list[q] > mine;
  // sorted, then each lane takes its rank's
  if (lane < found) list[place] = mine;
  const uint64_t k = lane < found ? list[lane] : 0;
  my_id = lane < top_k ? key_expert(k) : -1;
  my_logit = lane < top_k ? key_logit(k) : 0.f;
  top_logit = key_logit(list[0]);
}

// One window of 512 values of a weight row and of a token's row, as in the
// streaming product: lane group g takes block 4 i + g at step i.
struct WeightWindow {
  dwords4 w[4], s;
};

struct Weights {
  __amdgpu_buffer_rsrc_t codes, scales;
  uint32_t at, scales_at;  // this lane's row
  int blocks;
};

__device__ __forceinline__ void load_window(WeightWindow& b, const Weights& w, int win) {
  const int g = (threadIdx.x & 63) >> 4, b0 = win * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int blk = b0 + 4 * i + g;
    b.w[i] = buffer_load16(w.codes, blk < w.blocks ? w.at + blk * 16 : kOutOfRange);
  }
  if (b0 + 12 < w.blocks) {
    b.s = buffer_load16(w.scales, w.scales_at + b0);
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      b.s[i] = buffer_load4(w.scales, b0 + 4 * i < w.blocks ? w.scales_at + b0 + 4 * i : kOutOfRange);
  }
}

// acc += the window's products; row(i, blk) gives the token's block of step i,
// word(i, blk) the scale word that holds blocks blk ... blk + 3.
template <typename Row, typename Word>
__device__ __forceinline__ void multiply_window(f32x4& acc, const WeightWindow& b, int win,
                                                int blocks, Row&& row, Word&& word) {
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int blk = win * 16 + 4 * i;
    if (blk >= blocks) return;
    const bool in = blk + g < blocks;  // blocks behind K are zeros of scale 1
    const uint32_t sw = in ? b.s[i] >> (8 * g) : 127u;
    const uint32_t sa = in ? word(i, blk) >> (8 * g) : 127u;
    const dwords4 a = in ? row(i, blk + g) : dwords4{};
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(b.w[i]), operand(a), acc, kFp4,
                                                           kFp4, 0, sw, 0, sa);
  }
}

constexpr int kInFlight = 2;  // windows; four or six are slower (22.2, 22.6 against 21.1 us)

// ---- gate/up -------------------------------------------------------------------
// K is shared out to the waves in windows, kParts fours of waves per workgroup: one
// or four shares cost one token half a microsecond, four shares four tokens ten.
constexpr int kParts = 2, kWaves = 4 * kParts;
constexpr int kQuantWords = 2;  // words per lane whose loads are in flight (six tokens: 67 us with one)

template <int NPL, typename TX>
__global__ __launch_bounds__(64 * kWaves) void small_gate_up_kernel(MxSmallArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  __shared__ int ids[kMaxSlots];
  __shared__ uint64_t lists[kMaxTokens][64];
  __shared__ float h[kWaves][16][17];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int S = p.T * p.top_k;
  const int n_tiles = p.I / 32;
  const int mt = blockIdx.x / n_tiles, nt = blockIdx.x - mt * n_tiles;
  const int blocks = p.H / 32, sbytes = mx_scale_bytes(p.H);
  uint8_t* codes = lds;                        // [T, H / 2]
  uint8_t* scales = lds + p.T * (p.H / 2);     // [T, sbytes]

  if (wave < p.T) {
    int id;
    float logit, top;
    small_topk<NPL>(p.logits + static_cast<size_t>(wave) * p.E, p.E, p.top_k, lists[wave], id,
                    logit, top);
    const float w = wave_topk_weight(logit, top, p.top_k);
    if (lane < p.top_k) {
      const int s = wave * p.top_k + lane;
      ids[s] = id;
      if (blockIdx.x == 0) {
        p.ids[s] = id;
        p.weights[s] = w;
      }
    }
  }
  // the waves without a token to route quantise them
  const int q0 = p.T;
  static_assert(kWaves > kMaxTokens, "some wave quantises");
  if (wave >= q0) {
    const int words = p.H / 8, total = p.T * words, step = (kWaves - q0) * 64;
    for (int i0 = (wave - q0) * 64; i0 < total; i0 += step * kQuantWords) {
      float v[kQuantWords][8];
      int t[kQuantWords], c[kQuantWords];
#pragma unroll
      for (int u = 0; u < kQuantWords; ++u) {
        const int i = min(i0 + u * step + lane, total - 1);  // whole blocks: total is a multiple of 4
        t[u] = i / words, c[u] = i - t[u] * words;
        load8<TX>(
            static_cast<const typename TX::bits*>(p.x) + static_cast<size_t>(t[u]) * p.H + 8 * c[u], 8,
            v[u]);
      }
#pragma unroll
      for (int u = 0; u < kQuantWords; ++u) {
        uint32_t m = 0;
#pragma unroll
        for (int q = 0; q < 8; ++q) m = max(m, abs_bits(v[u][q]));
        m = quad_max<0xB1>(m);
        m = quad_max<0x4E>(m);
        const uint32_t byte = mx_scale_byte(m);
        if (i0 + u * step + lane < total) {
          *reinterpret_cast<uint32_t*>(codes + t[u] * (p.H / 2) + 4 * c[u]) = mx_word(v[u], byte);
          if ((c[u] & 3) == 0) scales[t[u] * sbytes + (c[u] >> 2)] = static_cast<uint8_t>(byte);
        }
      }
    }
  }
  __syncthreads();

  const int id = lane < S ? ids[lane] : INT32_MAX;
  const Places at = place_slots(id, S);
  const unsigned long long mine = slots_of(at, S, mt);
  if (mine == 0) return;  // fewer active experts: the whole workgroup alike
  const int lead = __builtin_ctzll(mine);
  const int e = __builtin_amdgcn_readlane(id, lead), r0 = __builtin_amdgcn_readlane(at.row, lead);
  const int rows = __popcll(mine);

  const int col = lane & 15;
  const int n = ((wave >> 1) & 1) * p.I + nt * 32 + (wave & 1) * 16 + col;
  const int part = wave >> 2;
  const int64_t N = 2 * static_cast<int64_t>(p.I);
  const Weights w{make_rsrc(p.w13_codes + e * N * (p.H / 2), static_cast<uint32_t>(N) * (p.H / 2)),
                  make_rsrc(p.w13_scales + e * N * sbytes, static_cast<uint32_t>(N) * sbytes),
                  static_cast<uint32_t>(n) * (p.H / 2), static_cast<uint32_t>(n) * sbytes, blocks};
  // the token of the tile's row `col`: its slots hold the rows in order
  unsigned long long left = mine;
  for (int q = 0; q < col && left; ++q) left &= left - 1;
  const int token = left ? __builtin_ctzll(left) / p.top_k : -1;
  const uint8_t* my_codes = codes + max(token, 0) * (p.H / 2);
  const uint8_t* my_scales = scales + max(token, 0) * sbytes;
  auto row = [&](int, int blk) {
    return token >= 0 ? *reinterpret_cast<const dwords4*>(my_codes + blk * 16) : dwords4{};
  };
  auto word = [&](int, int blk) -> uint32_t {
    return token >= 0 ? *reinterpret_cast<const uint32_t*>(my_scales + blk) : 0x7F7F7F7Fu;
  };

  const int windows = (blocks + 15) / 16;
  WeightWindow b[kInFlight];
#pragma unroll
  for (int i = 0; i < kInFlight; ++i) load_window(b[i], w, part + i * kParts);
  f32x4 acc{};
  for (int win = part; win < windows; win += kInFlight * kParts) {
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      const int at = win + i * kParts;
      if (at < windows) multiply_window(acc, b[i], at, blocks, row, word);
      load_window(b[i], w, at + kInFlight * kParts);
    }
  }
  gate_up_epilogue<kParts>(acc, h, wave, p.I, nt, r0, rows, p.act_codes, p.act_scales);
}

// ---- down and combine --------------------------------------------------------------
// Without registers to spill: 16 waves are held to 128 each, and one token then
// takes 26 us instead of 18.6 (8 or 10 waves 18.6).
constexpr int kDownWaves = 12;

// A wave's windows of one expert after another are one sequence, two of them in
// flight with the rows they meet, so that no expert starts from an empty pipe.
struct DownExpert {
  Weights w;  // no blocks: none left, loads give zeros
  const uint8_t *codes, *scales;
  int r0, count;  // its rows
};
struct DownWindow {
  WeightWindow w;
  dwords4 a[4];
  uint32_t s[4];
};
__device__ __forceinline__ void load_window(DownWindow& b, const DownExpert& x, int win) {
  const int col = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
  load_window(b.w, x.w, win);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int blk = win * 16 + 4 * i;
    b.a[i] = dwords4{};
    b.s[i] = 127u * 0x01010101u;
    if (col >= x.count) continue;
    if (blk + g < x.w.blocks) b.a[i] = *reinterpret_cast<const dwords4*>(x.codes + (blk + g) * 16);
    if (blk < x.w.blocks) b.s[i] = *reinterpret_cast<const uint32_t*>(x.scales + blk);
  }
}

template <typename TO>
__global__ __launch_bounds__(64 * kDownWaves) void small_down_kernel(MxSmallArgs p) {
  __shared__ float y[kMaxSlots][17];
  __shared__ int rows_of[kMaxSlots];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int S = p.T * p.top_k;
  const int id = lane < S ? p.ids[lane] : INT32_MAX;
  const Places at = place_slots(id, S);
  if (wave == 0 && lane < S) rows_of[lane] = at.row;
  const int blocks = p.I / 32, sbytes = mx_scale_bytes(p.I);
  const int col = lane & 15, g = lane >> 4;
  const int n = blockIdx.x * 16 + col;
  const int windows = (blocks + 15) / 16;
  auto expert = [&](int x) {
    const unsigned long long mine = slots_of(at, S, x);
    const int lead = mine ? __builtin_ctzll(mine) : 0;
    const int e = mine ? __builtin_amdgcn_readlane(id, lead) : 0;
    DownExpert q;
    q.r0 = __builtin_amdgcn_readlane(at.row, lead);
    q.count = __popcll(mine);
    const int r = q.r0 + (col < q.count ? col : 0);
    q.w = {make_rsrc(p.w2_codes + static_cast<int64_t>(e) * p.H * (p.I / 2),
                     static_cast<uint32_t>(p.H) * (p.I / 2)),
           make_rsrc(p.w2_scales + static_cast<int64_t>(e) * p.H * sbytes,
                     static_cast<uint32_t>(p.H) * sbytes),
           static_cast<uint32_t>(n) * (p.I / 2), static_cast<uint32_t>(n) * sbytes,
           mine ? blocks : 0};
    q.codes = p.act_codes + static_cast<int64_t>(r) * (p.I / 2);
    q.scales = p.act_scales + static_cast<int64_t>(r) * sbytes;
    return q;
  };
  auto multiply = [&](f32x4& acc, const DownWindow& b, int win) {
    multiply_window(acc, b.w, win, blocks, [&](int i, int) { return b.a[i]; },
                    [&](int i, int) { return b.s[i]; });
  };
  DownExpert now = expert(wave);
  DownWindow b[2];
  load_window(b[0], now, 0);
  load_window(b[1], now, 1);
  for (int x = wave + kDownWaves; now.count > 0; x += kDownWaves) {
    const DownExpert next = expert(x);
    f32x4 acc{};
    int win = 0;
    for (; win + 2 < windows; win += 2) {
      multiply(acc, b[0], win);
      load_window(b[0], now, win + 2);
      multiply(acc, b[1], win + 1);
      load_window(b[1], now, win + 3);
    }
    multiply(acc, b[0], win);
    load_window(b[0], next, 0);
    multiply(acc, b[1], win + 1);  // nothing if there is none
    load_window(b[1], next, 1);
    if (col < now.count) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y[now.r0 + col][4 * g + i] = acc[i];
    }
    now = next;
  }
  __syncthreads();
  const int t = threadIdx.x >> 4, c = threadIdx.x & 15;
  if (t < p.T) {
    float sum = 0.f;
    for (int j = 0; j < p.top_k; ++j)
      sum = fmaf(p.weights[t * p.top_k + j], y[rows_of[t * p.top_k + j]][c], sum);
    static_cast<typename TO::bits*>(p.out)[static_cast<size_t>(t) * p.H + blockIdx.x * 16 + c] =
        from_float(TO{}, sum);
  }
}

template <int NPL, typename TX>
void launch_gate_up(const MxSmallArgs& p, hipStream_t stream) {
  const int S = p.T * p.top_k, active = p.E < S ? p.E : S;
  const size_t lds = static_cast<size_t>(p.T) * (p.H / 2 + mx_scale_bytes(p.H));
  hipLaunchKernelGGL((small_gate_up_kernel<NPL, TX>), dim3(active * (p.I / 32)), dim3(64 * kWaves), lds,
                     stream, p);
}

}  // namespace

bool mx_small_ok(int64_t T, int top_k, int E, int H, int I) {
  return T <= kMaxTokens && T * top_k <= kMaxSlots && E <= 1024 && H <= kMxSmallHidden && I > 0;
}

void launch_mx_small_layer(const MxSmallArgs& p, hipStream_t stream) {
  with_dtype(p.dtype, [&](auto t) {
    using T = decltype(t);
    if (p.E <= 64)
      launch_gate_up<1, T>(p, stream);
    else if (p.E <= 128)
      launch_gate_up<2, T>(p, stream);
    else if (p.E <= 256)
      launch_gate_up<4, T>(p, stream);
    else if (p.E <= 512)
      launch_gate_up<8, T>(p, stream);
    else
      launch_gate_up<16, T>(p, stream);
    hipLaunchKernelGGL(small_down_kernel<T>, dim3(p.H / 16), dim3(64 * kDownWaves), 0, stream, p);
  });
}

}  // namespace moe
