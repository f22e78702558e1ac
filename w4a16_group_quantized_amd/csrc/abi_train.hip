// C ABI of the training operators: argument validation and dispatch.
// Declarations and the full contract are in include/moe_w4a16.h.  Nothing here
// allocates, frees or synchronises.
#include "train.h"
#include "typed.h"

#include <math.h>

#include <algorithm>

namespace {

using namespace moe;

constexpr int kMaxColumns = 65536;
constexpr int64_t kMaxStride = static_cast<int64_t>(1) << 31;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
inline bool ok_typed(const void* p, int dtype) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % dtype_bytes(dtype) == 0;
}
int check_launch() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

int check_stride(int64_t cols, int64_t ld) {
  if (ld < cols) return MOE_ERR_INVALID_ARG;
  return ld > kMaxStride ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// The sizes that the three products share.
int check_grouped(int32_t dtype, int32_t out_dtype, int64_t rows, bool offsets, int32_t E, int32_t N,
                  int32_t K) {
  if (!dtype_ok(dtype) || !dtype_ok(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (rows < 0 || E < 1 || N < 1 || K < 1 || (!offsets && E != 1)) return MOE_ERR_INVALID_ARG;
  if (dtype == MOE_F32) return MOE_ERR_UNSUPPORTED;
  if (E > kMaxExperts || N > kMaxColumns || K > kMaxColumns) return MOE_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(N) * K >= (static_cast<int64_t>(1) << 30)) return MOE_ERR_UNSUPPORTED;
  if (rows > (1 << 27)) return MOE_ERR_UNSUPPORTED;
  // tiles are numbered with 31 bits
  const int64_t most = N > K ? N : K;
  const int64_t tiles = (rows / 16 + (E < rows ? E : rows)) * ((most + 63) / 64);
  return tiles >= (1 << 24) ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// The products of rows: `in` columns read, `cols` written.
int grouped_rows(Product p, const void* x, int32_t dtype, int64_t rows, int64_t x_stride,
                 const int32_t* offsets, int32_t E, const void* w, int32_t N, int32_t K, void* out,
                 int32_t out_dtype, int64_t out_stride, void* stream) {
  if (int st = check_grouped(dtype, out_dtype, rows, offsets != nullptr, E, N, K)) return st;
  const int32_t in = p == Product::kOut ? K : N, cols = p == Product::kOut ? N : K;
  if (int st = check_stride(in, x_stride)) return st;
  if (int st = check_stride(cols, out_stride)) return st;
  if (rows == 0) return MOE_OK;
  if (!ok_typed(x, dtype) || !ok_ptr(w) || !aligned16(offsets) || !ok_typed(out, out_dtype))
    return MOE_ERR_INVALID_ARG;
  GroupedArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.x_ld = x_stride;
  a.y = static_cast<const uint16_t*>(w);
  a.dtype = dtype;
  a.offsets = offsets;
  a.rows = static_cast<int>(rows);
  a.E = E;
  a.N = N;
  a.K = K;
  a.out = out;
  a.out_dtype = out_dtype;
  a.out_ld = out_stride;
  launch_grouped(p, a, static_cast<hipStream_t>(stream));
  return check_launch();
}

int check_act(int32_t dtype, int64_t rows, int32_t I, const int32_t* offsets, int32_t E) {
  if (!dtype_ok(dtype) || rows < 0 || I < 1) return MOE_ERR_INVALID_ARG;
  if (offsets != nullptr && E < 1) return MOE_ERR_INVALID_ARG;
  if (I > kMaxColumns / 2 || rows > INT32_MAX || (offsets != nullptr && E > kMaxExperts))
    return MOE_ERR_UNSUPPORTED;
  // one thread per 8 columns, numbered with 32 bits
  return rows * ((I + 7) / 8) >= (static_cast<int64_t>(1) << 32) - 256 ? MOE_ERR_UNSUPPORTED : MOE_OK;
}

// f(address, bytes) for each buffer that an AdamW step writes.
template <typename F>
void adamw_written(const moe_adamw_tensor* tensors, int32_t count, int32_t state_bits, F&& f) {
  const auto put = [&](const void* p, uint64_t bytes) { f(reinterpret_cast<uint64_t>(p), bytes); };
  for (int32_t i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (t.n == 0) continue;
    const uint64_t n = static_cast<uint64_t>(t.n), blocks = (n + kAdamwBlock - 1) / kAdamwBlock;
    put(t.param, n * dtype_bytes(t.param_dtype));
    put(t.m, n * (state_bits / 8));
    put(t.v, n * (state_bits / 8));
    if (state_bits == 8) {
      put(t.m_scales, blocks * sizeof(float));
      put(t.v_scales, blocks * sizeof(float));
    }
    if (t.copy != nullptr) put(t.copy, n * dtype_bytes(t.copy_dtype));
  }
}

// And for each that it only reads.
template <typename F>
void adamw_read(const moe_adamw_tensor* tensors, int32_t count, const float* grad_scale, F&& f) {
  for (int32_t i = 0; i < count; ++i)
    if (tensors[i].n > 0)
      f(reinterpret_cast<uint64_t>(tensors[i].grad),
        static_cast<uint64_t>(tensors[i].n) * dtype_bytes(tensors[i].grad_dtype));
  if (grad_scale != nullptr) f(reinterpret_cast<uint64_t>(grad_scale), uint64_t{sizeof(float)});
}

// Whether every buffer that the step writes is apart from all others of the call.  Written
// ranges are held kHeld at a time, on the stack: they are apart from each other when their
// sorted beginnings and ends take turns, and then each of the rest is looked up among them.
int check_apart(const moe_adamw_tensor* tensors, int32_t count, int32_t state_bits,
                const float* grad_scale) {
  constexpr size_t kHeld = 2048;  // 32 KB; 340 tensors with 8-bit states and copies
  uint64_t begins[kHeld], ends[kHeld];
  for (size_t first = 0, all = 1; first < all; first += kHeld) {
    size_t n = 0;
    all = 0;
    adamw_written(tensors, count, state_bits, [&](uint64_t from, uint64_t bytes) {
      if (all >= first && n < kHeld) {
        begins[n] = from;
        ends[n++] = from + bytes;
      }
      ++all;
    });
    std::sort(begins, begins + n);
    std::sort(ends, ends + n);
    bool apart = true;
    for (size_t i = 1; i < n; ++i) apart = apart && ends[i - 1] <= begins[i];
    if (!apart) return MOE_ERR_INVALID_ARG;
    const auto look_up = [&](uint64_t from, uint64_t bytes) {
      const size_t next = std::upper_bound(ends, ends + n, from) - ends;
      apart = apart && (next == n || from + bytes <= begins[next]);
    };
    size_t at = 0;
    if (first + n < all)
      adamw_written(tensors, count, state_bits, [&](uint64_t from, uint64_t bytes) {
        if (at++ >= first + n) look_up(from, bytes);
      });
    adamw_read(tensors, count, grad_scale, look_up);
    if (!apart) return MOE_ERR_INVALID_ARG;
  }
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_grouped_gemm(const void* a, int32_t dtype, int64_t rows, int64_t a_stride,
                     const int32_t* expert_offsets, int32_t E, const void* w, int32_t N, int32_t K,
                     void* out, int32_t out_dtype, int64_t out_stride, void* stream) {
  return grouped_rows(Product::kOut, a, dtype, rows, a_stride, expert_offsets, E, w, N, K, out,
                      out_dtype, out_stride, stream);
}

int moe_grouped_gemm_backward(const void* grad, int32_t dtype, int64_t rows, int64_t grad_stride,
                              const int32_t* expert_offsets, int32_t E, const void* w, int32_t N,
                              int32_t K, void* grad_a, int32_t out_dtype, int64_t grad_a_stride,
                              void* stream) {
  return grouped_rows(Product::kRows, grad, dtype, rows, grad_stride, expert_offsets, E, w, N, K,
                      grad_a, out_dtype, grad_a_stride, stream);
}

size_t moe_grouped_gemm_backward_weights_workspace_bytes(int64_t rows, int32_t E, int32_t N,
                                                         int32_t K) {
  if (check_grouped(MOE_BF16, MOE_F32, rows, true, E, N, K) != MOE_OK) return 0;
  return grouped_workspace_bytes(rows, E, N, K);
}

int moe_grouped_gemm_backward_weights(const void* grad, int32_t dtype, int64_t rows,
                                      int64_t grad_stride, const void* a, int64_t a_stride,
                                      const int32_t* expert_offsets, int32_t E, int32_t N,
                                      int32_t K, void* grad_w, int32_t out_dtype,
                                      int32_t accumulate, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  if (int st = check_grouped(dtype, out_dtype, rows, expert_offsets != nullptr, E, N, K)) return st;
  if (accumulate != 0 && accumulate != 1) return MOE_ERR_INVALID_ARG;
  if (int st = check_stride(N, grad_stride)) return st;
  if (int st = check_stride(K, a_stride)) return st;
  if (!ok_ptr(grad_w) || !aligned16(expert_offsets)) return MOE_ERR_INVALID_ARG;
  if (rows > 0 && (!ok_typed(grad, dtype) || !ok_typed(a, dtype))) return MOE_ERR_INVALID_ARG;
  const size_t need = grouped_workspace_bytes(rows, E, N, K);
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  if (need > 0 && !ok_ptr(workspace)) return MOE_ERR_INVALID_ARG;
  GroupedArgs p{};
  p.x = static_cast<const uint16_t*>(grad);
  p.x_ld = grad_stride;
  p.y = static_cast<const uint16_t*>(a);
  p.y_ld = a_stride;
  p.dtype = dtype;
  p.offsets = expert_offsets;
  p.rows = static_cast<int>(rows);
  p.E = E;
  p.N = N;
  p.K = K;
  p.out = grad_w;
  p.out_dtype = out_dtype;
  p.accumulate = accumulate;
  p.partial = static_cast<float*>(workspace);
  launch_grouped(Product::kWeights, p, static_cast<hipStream_t>(stream));
  return check_launch();
}

int moe_silu_mul(const void* h, int32_t dtype, int64_t rows, int32_t I, int64_t h_stride,
                 const int32_t* expert_offsets, int32_t E, void* act, int64_t act_stride,
                 void* stream) {
  if (int st = check_act(dtype, rows, I, expert_offsets, E)) return st;
  if (int st = check_stride(2 * static_cast<int64_t>(I), h_stride)) return st;
  if (int st = check_stride(I, act_stride)) return st;
  if (rows == 0) return MOE_OK;
  if (!ok_typed(h, dtype) || !ok_typed(act, dtype) || !aligned16(expert_offsets))
    return MOE_ERR_INVALID_ARG;
  ActArgs a{};
  a.h = h;
  a.h_ld = h_stride;
  a.dtype = dtype;
  a.rows = static_cast<int>(rows);
  a.I = I;
  a.offsets = expert_offsets;
  a.E = E;
  a.out = act;
  a.out_ld = act_stride;
  launch_silu_mul(a, false, static_cast<hipStream_t>(stream));
  return check_launch();
}

int moe_silu_mul_backward(const void* grad_act, int64_t grad_stride, const void* h,
                          int64_t h_stride, int32_t dtype, int64_t rows, int32_t I,
                          const int32_t* expert_offsets, int32_t E, void* grad_h,
                          int64_t grad_h_stride, void* stream) {
  if (int st = check_act(dtype, rows, I, expert_offsets, E)) return st;
  if (int st = check_stride(I, grad_stride)) return st;
  if (int st = check_stride(2 * static_cast<int64_t>(I), h_stride)) return st;
  if (int st = check_stride(2 * static_cast<int64_t>(I), grad_h_stride)) return st;
  if (rows == 0) return MOE_OK;
  if (!ok_typed(grad_act, dtype) || !ok_typed(h, dtype) || !ok_typed(grad_h, dtype) ||
      !aligned16(expert_offsets))
    return MOE_ERR_INVALID_ARG;
  ActArgs a{};
  a.grad = grad_act;
  a.grad_ld = grad_stride;
  a.h = h;
  a.h_ld = h_stride;
  a.dtype = dtype;
  a.rows = static_cast<int>(rows);
  a.I = I;
  a.offsets = expert_offsets;
  a.E = E;
  a.out = grad_h;
  a.out_ld = grad_h_stride;
  launch_silu_mul(a, true, static_cast<hipStream_t>(stream));
  return check_launch();
}

int moe_route_backward(const int32_t* topk_ids, const float* topk_weights,
                       const float* grad_weights, int64_t T, int32_t E, int32_t top_k,
                       void* grad_logits, int32_t out_dtype, void* stream) {
  if (!dtype_ok(out_dtype) || T < 0 || E < 1 || top_k < 1) return MOE_ERR_INVALID_ARG;
  // a wave per token, in workgroups of four, and less than 2^32 threads in a launch
  if (E > kMaxExperts || top_k > kMaxTopK || T > (1 << 26) - 4 || T * top_k > INT32_MAX)
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!ok_ptr(topk_ids) || !ok_ptr(topk_weights) || !ok_ptr(grad_weights) || !ok_ptr(grad_logits))
    return MOE_ERR_INVALID_ARG;
  launch_route_backward(topk_ids, topk_weights, grad_weights, static_cast<int>(T), E, top_k,
                        grad_logits, out_dtype, static_cast<hipStream_t>(stream));
  return check_launch();
}

int moe_adamw(const moe_adamw_tensor* tensors, int32_t count, int32_t state_bits, double lr,
              double beta1, double beta2, double eps, double weight_decay, int64_t step,
              uint32_t seed, const float* grad_scale, void* stream) {
  if (count < 0 || (count > 0 && tensors == nullptr)) return MOE_ERR_INVALID_ARG;
  if (state_bits != 8 && state_bits != 32) return MOE_ERR_INVALID_ARG;
  // written so that a NaN is refused too
  if (!(lr >= 0) || !(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1) || !(eps >= 0) ||
      !(weight_decay >= 0) || step < 1 || isinf(lr) || isinf(eps) || isinf(weight_decay))
    return MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(grad_scale) % 4) return MOE_ERR_INVALID_ARG;
  bool any = false;
  for (int32_t i = 0; i < count; ++i) {
    const moe_adamw_tensor& t = tensors[i];
    if (!dtype_ok(t.param_dtype) || !dtype_ok(t.grad_dtype) || t.n < 0) return MOE_ERR_INVALID_ARG;
    if (t.n > (static_cast<int64_t>(1) << 33)) return MOE_ERR_UNSUPPORTED;
    if (t.n == 0) continue;
    any = true;
    if (!ok_typed(t.param, t.param_dtype) || !ok_typed(t.grad, t.grad_dtype))
      return MOE_ERR_INVALID_ARG;
    if (t.copy != nullptr && (!dtype_ok(t.copy_dtype) || !ok_typed(t.copy, t.copy_dtype)))
      return MOE_ERR_INVALID_ARG;
    if (state_bits == 32) {
      if (!ok_typed(t.m, MOE_F32) || !ok_typed(t.v, MOE_F32)) return MOE_ERR_INVALID_ARG;
    } else if (t.m == nullptr || t.v == nullptr || !ok_typed(t.m_scales, MOE_F32) ||
               !ok_typed(t.v_scales, MOE_F32)) {
      return MOE_ERR_INVALID_ARG;
    }
  }
  if (!any) return MOE_OK;
  if (int st = check_apart(tensors, count, state_bits, grad_scale)) return st;
  AdamwScalars s;
  s.beta1 = static_cast<float>(beta1);
  s.rest1 = static_cast<float>(1 - beta1);
  s.beta2 = static_cast<float>(beta2);
  s.rest2 = static_cast<float>(1 - beta2);
  s.decay = static_cast<float>(lr * weight_decay);
  s.size = static_cast<float>(lr / (1 - pow(beta1, static_cast<double>(step))));
  if (isinf(s.decay) || isinf(s.size)) return MOE_ERR_INVALID_ARG;
  s.root = static_cast<float>(1 / sqrt(1 - pow(beta2, static_cast<double>(step))));
  // a positive eps stays positive: an element without moments moves by 0 / eps = 0
  s.eps = eps > 0 ? fmaxf(static_cast<float>(eps), 0x1p-149f) : 0.f;
  s.grad_scale = grad_scale;
  s.seed = seed;
  s.small = ldexp(static_cast<double>(s.root), -63) > ldexp(static_cast<double>(s.eps), -25);
  launch_adamw(tensors, count, state_bits, s, static_cast<hipStream_t>(stream));
  return check_launch();
}

}  // extern "C"
