// What a training step needs between the experts' products and around the router:
//   act            = gate s up,  s = 1 / (1 + e^-gate),  of h = [gate | up]
//   grad of gate   = grad up s (1 + gate (1 - s)),  grad of up = grad gate s
//   grad of logits = w_j (g_j - sum_i w_i g_i) at the chosen experts, 0 elsewhere
// (w the softmax over a token's chosen logits, g the gradient of w).  All are bound
// by memory; arithmetic is fp32, rounded once at the store.  40960 rows, I = 640, bf16:
// activation 29 us (5.4 TB/s), its gradient 45 (5.8); 40957 rows, I = 641, whose rows
// begin at any element, 32 and 47; fp32 49 and 86 (6.4 and 6.1 TB/s).  80 rows 3.0 us.
// The router's gradient of 4096 tokens, 512 experts, 10 each: 5.7 us, 8 tokens 2.9.
#include "train.h"
#include "typed.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// s = 1 / (1 + e^-x) and 1 - s, both without cancellation: with z = e^-|x| they are
// 1 / (1 + z) and z / (1 + z) in one order or the other.  The exponential is that of
// 2^t (1 + r ln 2) with t = -|x| log2(e) rounded and r what that rounding left (2
// units in the last place); |x| is held below 128, where z is 0 already, so that r
// stays finite.  A z under 2^-126 counts as 0.  A NaN goes through the caller's
// products with x.
__device__ __forceinline__ void sigmoid(float x, float& s, float& rest) {
  constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f, kLn2 = 0.693147181f;
  const float a = -fminf(fabsf(x), 128.f);
  const float t = a * kLog2e;
  const float r = fmaf(a, kLog2eRest, fmaf(a, kLog2e, -t));
  const float z = __builtin_amdgcn_exp2f(t) * fmaf(r, kLn2, 1.f);
  const float big = __builtin_amdgcn_rcpf(1.f + z), small = z * big;
  s = x >= 0.f ? big : small;
  rest = x >= 0.f ? small : big;
}

// 8 columns of a row per thread.
template <typename T, bool BACKWARD>
__global__ __launch_bounds__(kThreads) void silu_mul_kernel(ActArgs p) {
  using B = typename T::bits;
  const int units = (p.I + 7) / 8;
  // the block's first unit by one division; its threads' rows by 32-bit ones
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kThreads;
  const int64_t row0 = first / units;
  const uint32_t u = static_cast<uint32_t>(first - row0 * units) + threadIdx.x;
  const int64_t row = row0 + u / static_cast<uint32_t>(units);
  const int c = static_cast<int>(u % static_cast<uint32_t>(units)) * 8;
  if (row >= p.rows) return;
  if (p.offsets != nullptr && (row < p.offsets[0] || row >= p.offsets[p.E])) return;
  const int n = p.I - c;
  const B* h = static_cast<const B*>(p.h) + row * p.h_ld + c;
  float gate[8], up[8];
  load8<T>(h, n, gate);
  load8<T>(h + p.I, n, up);
  B* out = static_cast<B*>(p.out) + row * p.out_ld + c;
  if constexpr (!BACKWARD) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s, rest;
      sigmoid(gate[i], s, rest);
      gate[i] *= s * up[i];
    }
    store8<T>(out, n, gate);
  } else {
    float grad[8];
    load8<T>(static_cast<const B*>(p.grad) + row * p.grad_ld + c, n, grad);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s, rest;
      sigmoid(gate[i], s, rest);
      const float gs = grad[i] * s;
      grad[i] = gs * up[i] * fmaf(gate[i], rest, 1.f);
      up[i] = gs * gate[i];
    }
    store8<T>(out, n, grad);
    store8<T>(out + p.I, n, up);
  }
}

// One wave per token.  Lane j holds choice j; a lane's 8 columns are compared with
// every choice, so an expert that a token names twice gets the sum of both.
template <typename TO>
__global__ __launch_bounds__(kThreads) void route_backward_kernel(
    const int* __restrict__ ids, const float* __restrict__ weights, const float* __restrict__ grad,
    int T, int E, int top_k, typename TO::bits* __restrict__ out) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6);
  if (t >= T) return;
  const int64_t at = static_cast<int64_t>(t) * top_k + lane;
  int id = -1;
  float w = 0.f, g = 0.f;
  if (lane < top_k) {
    id = ids[at];
    w = weights[at];
    g = grad[at];
  }
  float dot = w * g;
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d, 64);
  const float each = w * (g - dot);
  for (int c0 = 0; c0 < E; c0 += 64 * 8) {  // all lanes: each holds a choice that others read
    const int c = c0 + lane * 8;
    float v[8] = {};
    for (int j = 0; j < top_k; ++j) {
      const int to = __builtin_amdgcn_readlane(id, j) - c;
      const float x = __builtin_bit_cast(
          float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, each), j));
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] += to == i ? x : 0.f;
    }
    if (c < E) store8<TO>(out + static_cast<int64_t>(t) * E + c, E - c, v);
  }
}

}  // namespace

void launch_silu_mul(const ActArgs& a, bool backward, hipStream_t stream) {
  const int64_t units = static_cast<int64_t>(a.rows) * ((a.I + 7) / 8);
  const dim3 grid(static_cast<unsigned>((units + kThreads - 1) / kThreads));
  with_dtype(a.dtype, [&](auto t) {
    using T = decltype(t);
    if (backward)
      hipLaunchKernelGGL((silu_mul_kernel<T, true>), grid, dim3(kThreads), 0, stream, a);
    else
      hipLaunchKernelGGL((silu_mul_kernel<T, false>), grid, dim3(kThreads), 0, stream, a);
  });
}

void launch_route_backward(const int* ids, const float* weights, const float* grad, int T, int E,
                           int top_k, void* out, int out_dtype, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((T + kThreads / 64 - 1) / (kThreads / 64)));
  with_dtype(out_dtype, [&](auto to) {
    using TO = decltype(to);
    hipLaunchKernelGGL((route_backward_kernel<TO>), grid, dim3(kThreads), 0, stream, ids, weights,
                       grad, T, E, top_k, static_cast<typename TO::bits*>(out));
  });
}

}  // namespace moe
