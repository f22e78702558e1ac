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

namespace moe {
namespace {

// ---------------------------------------------------------------- streaming --
// Few rows per expert: bound by reading each active expert's weights once.
// A wave takes 16 weight rows over all of K, straight from memory to
// registers in windows of 512 values (a row's 256 bytes of codes and 16 bytes
// of scales), two windows in flight; the up to 16 tokens of its tile come
// through the caches.  Four waves make a workgroup: 64 output columns, or the
// two halves of gate and up of 32 columns of I.
constexpr int kTokens = 16;

struct Window {
  dwords4 w[4], a[4];
  dwords4 ws, as;
};

template <bool GATE_UP, typename TO>
__global__ __launch_bounds__(256) void mx_stream_kernel(MxGemmArgs p, int n_tiles) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int mt = blockIdx.x / n_tiles, nt = blockIdx.x - mt * n_tiles;
  int e, r0, r1;
  if (!find_tile(p.offsets, p.E, p.rows, kTokens, mt, e, r0, r1)) return;

  const int blocks = p.K / 32;  // 32-value blocks per row
  const int sbytes = mx_scale_bytes(p.K);
  const int col = lane & 15, g = lane >> 4;
  const int I = p.N / 2;
  const int n = GATE_UP ? (wave >> 1) * I + nt * 32 + (wave & 1) * 16 + col
                        : nt * 64 + wave * 16 + col;
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
  load(b0, 0);
  load(b1, 1);
  for (int w = 0; w < windows; w += 2) {
    compute(b0, w);
    load(b0, w + 2);
    if (w + 1 < windows) compute(b1, w + 1);
    load(b1, w + 3);
  }

  // acc[i] is column n0 + 4 g + i of token r0 + col
  if constexpr (!GATE_UP) {
    if (row >= r1) return;
    const int n0 = nt * 64 + wave * 16 + 4 * g;
    auto* o = static_cast<typename TO::bits*>(p.out) + row * p.out_ld + n0;
    store4<TO>(o, p.N - n0, acc);
  } else {
    __shared__ float h[4][kTokens][17];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[wave][col][4 * g + i] = acc[i];
    __syncthreads();
    // 16 threads per token, two neighbouring columns each
    const int t = threadIdx.x >> 4, c = (threadIdx.x & 15) * 2;
    float a[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const float gate = h[c >> 4][t][(c & 15) + q], up = h[2 + (c >> 4)][t][(c & 15) + q];
      a[q] = silu_mul(gate, up);
    }
    uint32_t m = max(abs_bits(a[0]), abs_bits(a[1]));
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(m, d, 16)));
    const uint32_t byte = mx_scale_byte(m);
    uint32_t q = mx_pair(a[0], a[1], byte);
    q |= __shfl_xor(q, 1, 16) << 8;  // valid in even threads
    q |= __shfl_xor(q, 2, 16) << 16; // valid in every fourth
    const int out_row = r0 + t;
    if (out_row < r1) {
      const int sb = mx_scale_bytes(I);
      if ((threadIdx.x & 3) == 0)
        *reinterpret_cast<uint32_t*>(p.act_codes + static_cast<int64_t>(out_row) * (I / 2) +
                                     nt * 16 + c / 2) = q;
      if ((threadIdx.x & 15) == 0)
        store_scale(p.act_scales + static_cast<int64_t>(out_row) * sb, nt, I / 32, sb, byte);
    }
  }
}

}  // namespace

void launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream) {
  const bool gate_up = a.act_codes != nullptr;
  const int n_tiles = gate_up ? a.N / 64 : (a.N + 63) / 64;
  // an expert's last tile may be partial: at most one more tile per expert
  const int m_tiles = a.rows / kTokens + (a.E < a.rows ? a.E : a.rows);
  const dim3 grid(static_cast<unsigned>(m_tiles) * n_tiles);
  if (gate_up) {
    hipLaunchKernelGGL((mx_stream_kernel<true, F32>), grid, dim3(256), 0, stream, a, n_tiles);
    return;
  }
  with_dtype(a.out_dtype, [&](auto t) {
    using T = decltype(t);
    hipLaunchKernelGGL((mx_stream_kernel<false, T>), grid, dim3(256), 0, stream, a, n_tiles);
  });
}

}  // namespace moe
