// Token rows to expert order and back, with their gradients.  slot_rows[s] is
// the row of slot s = t * top_k + j in expert order; a value outside
// [0, rows) marks a slot that was left out.
//
//   dispatch           out[slot_rows[s], :] = x[s / top_k, :]
//   its gradient       the combine below without weights
//   combine            out[t, :] = sum_j w[t, j] y[slot_rows[t, j], :], j ascending
//   combine backward   grad_y[slot_rows[s], :] = w[s] grad[t, :]
//                      grad_w[s] = sum_h grad[t, h] y[slot_rows[s], h]   (0: left out)
//
// All are bound by memory.  Rows move in 16-byte accesses at any alignment;
// sums are fp32 in a fixed order, so a repeated call gives identical bits.
// Rows that no slot points at are neither read nor written.  4096 tokens x 10 x
// 2560 bf16, a tenth of the tokens without experts: dispatch 38 us (5.5 TB/s),
// combine 43 (4.9), combine backward 82 (4.9); 1021 tokens in fp32, dispatch
// backward 18.6 us (5.6).
#include "mxfp4.h"
#include "typed.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
// Rows of y whose loads are in flight together: more of them take registers that
// hide less than the waves they keep out (4096 tokens x 10 x 2560 bf16: 43 us with
// 4, 45 with 5, 54 with 8).
constexpr int kRowsInFlight = 4;
constexpr int64_t kMaxBlocks = 1 << 22;

dim3 blocks_for(int64_t items) {
  const int64_t n = (items + kThreads - 1) / kThreads;
  return dim3(static_cast<unsigned>(n < kMaxBlocks ? n : kMaxBlocks));
}

// One 16-byte unit of a token per thread, read once and written top_k times.
template <typename B>
__global__ __launch_bounds__(kThreads) void dispatch_kernel(
    const B* __restrict__ x, int T, int top_k, int H, int64_t x_ld,
    const int* __restrict__ slot_rows, B* __restrict__ out, int64_t out_ld, int rows) {
  constexpr int E = 16 / sizeof(B);
  const int units = (H + E - 1) / E;
  const int64_t total = static_cast<int64_t>(T) * units;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int t = static_cast<int>(i / units);
    const int c = static_cast<int>(i - static_cast<int64_t>(t) * units) * E;
    const B* src = x + t * x_ld + c;
    const int64_t s0 = static_cast<int64_t>(t) * top_k;
    const bool whole = c + E <= H;
    dwords4 d{};
    B e[E];
    if (whole) {
      d = load16(src);
    } else {
#pragma unroll
      for (int q = 0; q < E; ++q) e[q] = c + q < H ? src[q] : B{0};
    }
    for (int j0 = 0; j0 < top_k; j0 += kRowsInFlight) {
      int r[kRowsInFlight];
#pragma unroll
      for (int j = 0; j < kRowsInFlight; ++j) r[j] = j0 + j < top_k ? slot_rows[s0 + j0 + j] : -1;
#pragma unroll
      for (int j = 0; j < kRowsInFlight; ++j) {
        if (static_cast<uint32_t>(r[j]) >= static_cast<uint32_t>(rows)) continue;
        B* dst = out + r[j] * out_ld + c;
        if (whole) {
          store16(dst, d);
        } else {
#pragma unroll
          for (int q = 0; q < E; ++q)
            if (c + q < H) dst[q] = e[q];
        }
      }
    }
  }
}

// 8 columns of a token per thread; the loads of up to kRowsInFlight rows are in
// flight together.  A left-out slot adds nothing, whatever its weight holds.
template <typename TY, typename TO>
__global__ __launch_bounds__(kThreads) void combine_typed_kernel(
    const typename TY::bits* __restrict__ y, int T, int top_k, int H, int64_t y_ld,
    const float* __restrict__ weights, const int* __restrict__ slot_rows, int rows,
    typename TO::bits* __restrict__ out, int64_t out_ld) {
  const int units = (H + 7) / 8;
  const int64_t total = static_cast<int64_t>(T) * units;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kThreads) {
    const int t = static_cast<int>(i / units);
    const int c = static_cast<int>(i - static_cast<int64_t>(t) * units) * 8;
    const int n = H - c;
    const int64_t s0 = static_cast<int64_t>(t) * top_k;
    float acc[8] = {};
    for (int j0 = 0; j0 < top_k; j0 += kRowsInFlight) {
      int r[kRowsInFlight];
      float w[kRowsInFlight];
#pragma unroll
      for (int j = 0; j < kRowsInFlight; ++j) {
        const bool in = j0 + j < top_k;
        r[j] = in ? slot_rows[s0 + j0 + j] : -1;
        w[j] = weights == nullptr ? 1.f : (in ? weights[s0 + j0 + j] : 0.f);
      }
      float v[kRowsInFlight][8];
#pragma unroll
      for (int j = 0; j < kRowsInFlight; ++j) {
        const bool on = static_cast<uint32_t>(r[j]) < static_cast<uint32_t>(rows);
        if (on) load8<TY>(y + r[j] * y_ld + c, n, v[j]);
      }
#pragma unroll
      for (int j = 0; j < kRowsInFlight; ++j) {
        const bool on = static_cast<uint32_t>(r[j]) < static_cast<uint32_t>(rows);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[q] = on ? fmaf(w[j], v[j][q], acc[q]) : acc[q];
      }
    }
    store8<TO>(out + t * out_ld + c, n, acc);
  }
}

// One wave per slot: its row of y is read once, its row of grad_y written
// once; grad's row is read by the token's top_k waves, which sit in
// neighbouring workgroups and find it in L2.
template <typename TG, typename TY>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(
    const typename TG::bits* __restrict__ grad, int64_t grad_ld,
    const typename TY::bits* __restrict__ y, int64_t y_ld, const float* __restrict__ weights,
    const int* __restrict__ slot_rows, int64_t S, int top_k, int H, int rows,
    typename TY::bits* __restrict__ grad_y, int64_t grad_y_ld, float* __restrict__ grad_weights) {
  const int lane = threadIdx.x & 63;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kThreads / 64);
  for (int64_t s = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + (threadIdx.x >> 6); s < S;
       s += step) {
    const int r = slot_rows[s];
    float dot = 0.f;
    if (static_cast<uint32_t>(r) < static_cast<uint32_t>(rows)) {
      const float w = weights[s];
      const auto* g = grad + (s / top_k) * grad_ld;
      const auto* yr = y + r * y_ld;
      auto* dr = grad_y + r * grad_y_ld;
      // not unrolled: the waves hide the loads (4096 x 10 x 2560 bf16: 82 us; two
      // turns at a time 84, four 103)
#pragma unroll 1
      for (int c = lane * 8; c < H; c += 64 * 8) {
        float gv[8], yv[8];
        load8<TG>(g + c, H - c, gv);
        load8<TY>(yr + c, H - c, yv);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          dot = fmaf(gv[q], yv[q], dot);
          gv[q] *= w;
        }
        store8<TY>(dr + c, H - c, gv);
      }
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d, 64);
    if (lane == 0) grad_weights[s] = dot;
  }
}

}  // namespace

void launch_dispatch(const void* x, int bytes, int T, int top_k, int H, int64_t x_ld,
                     const int* slot_rows, void* out, int64_t out_ld, int rows,
                     hipStream_t stream) {
  const int E = 16 / bytes;
  const dim3 grid = blocks_for(static_cast<int64_t>(T) * ((H + E - 1) / E));
  if (bytes == 4)
    hipLaunchKernelGGL(dispatch_kernel<uint32_t>, grid, dim3(kThreads), 0, stream,
                       static_cast<const uint32_t*>(x), T, top_k, H, x_ld, slot_rows,
                       static_cast<uint32_t*>(out), out_ld, rows);
  else
    hipLaunchKernelGGL(dispatch_kernel<uint16_t>, grid, dim3(kThreads), 0, stream,
                       static_cast<const uint16_t*>(x), T, top_k, H, x_ld, slot_rows,
                       static_cast<uint16_t*>(out), out_ld, rows);
}

void launch_combine_typed(const void* y, int y_dtype, int T, int top_k, int H, int64_t y_ld,
                          const float* weights, const int* slot_rows, int rows, void* out,
                          int out_dtype, int64_t out_ld, hipStream_t stream) {
  const dim3 grid = blocks_for(static_cast<int64_t>(T) * ((H + 7) / 8));
  with_dtype(y_dtype, [&](auto ty) {
    with_dtype(out_dtype, [&](auto to) {
      using TY = decltype(ty);
      using TO = decltype(to);
      hipLaunchKernelGGL((combine_typed_kernel<TY, TO>), grid, dim3(kThreads), 0, stream,
                         static_cast<const typename TY::bits*>(y), T, top_k, H, y_ld, weights,
                         slot_rows, rows, static_cast<typename TO::bits*>(out), out_ld);
    });
  });
}

void launch_combine_backward(const void* grad, int grad_dtype, int64_t grad_ld, const void* y,
                             int y_dtype, int64_t y_ld, const float* weights,
                             const int* slot_rows, int T, int top_k, int H, int rows,
                             void* grad_y, int64_t grad_y_ld, float* grad_weights,
                             hipStream_t stream) {
  const int64_t S = static_cast<int64_t>(T) * top_k;
  const dim3 grid = blocks_for(S * 64);
  with_dtype(grad_dtype, [&](auto tg) {
    with_dtype(y_dtype, [&](auto ty) {
      using TG = decltype(tg);
      using TY = decltype(ty);
      hipLaunchKernelGGL((combine_backward_kernel<TG, TY>), grid, dim3(kThreads), 0, stream,
                         static_cast<const typename TG::bits*>(grad), grad_ld,
                         static_cast<const typename TY::bits*>(y), y_ld, weights, slot_rows, S,
                         top_k, H, rows, static_cast<typename TY::bits*>(grad_y), grad_y_ld,
                         grad_weights);
    });
  });
}

}  // namespace moe
