// C ABI of the MXFP4 operators and of the typed, masked token permutation:
// argument validation, workspace sizing and dispatch.  Declarations and the
// full contract are in include/moe_w4a16.h.  Nothing here allocates, frees or
// synchronises.
#include "mxfp4.h"
#include "typed.h"

namespace {

using namespace moe;

constexpr int kMaxK = 65536;
constexpr int kMaxColumns = 65536;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
// Typed tensors with a row stride need only their elements' alignment.
inline bool ok_typed(const void* p, int dtype) {
  return p != nullptr && reinterpret_cast<uintptr_t>(p) % dtype_bytes(dtype) == 0;
}
inline size_t align256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

int check_launch() {
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP;
}

// A strided matrix: rows that do not overlap, byte offsets within 63 bits.
int check_matrix(int64_t rows, int64_t cols, int64_t ld, int dtype) {
  if (!dtype_ok(dtype) || rows < 0 || ld < cols) return MOE_ERR_INVALID_ARG;
  if (ld > (static_cast<int64_t>(1) << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_mx(int64_t rows, int32_t K) {
  if (rows < 0 || K <= 0 || K % kGroup) return MOE_ERR_INVALID_ARG;
  if (K > kMaxK || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Slots of the typed permutation: any number of experts per token up to the
// limit (a token may hold fewer distinct ones than E).
int check_slots(int64_t T, int32_t top_k) {
  if (T < 0 || top_k < 1) return MOE_ERR_INVALID_ARG;
  // T by itself first: the product of a larger one could pass 64 bits
  if (top_k > kMaxTopK || T > INT32_MAX || T * top_k > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_rows(int64_t T, int32_t top_k, int32_t H, int64_t rows) {
  if (int st = check_slots(T, top_k)) return st;
  if (H <= 0 || rows < 0) return MOE_ERR_INVALID_ARG;
  if (H > kMaxColumns || rows > INT32_MAX) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int check_product(int64_t a_rows, int64_t rows, int32_t top_k, bool mapped, bool offsets,
                  int32_t E, int32_t N, int32_t K) {
  if (int st = check_mx(a_rows, K)) return st;
  if (rows < 0 || E < 1 || N < 1) return MOE_ERR_INVALID_ARG;
  if (mapped && top_k < 1) return MOE_ERR_INVALID_ARG;
  if (!mapped && rows > a_rows) return MOE_ERR_INVALID_ARG;
  if (!offsets && E != 1) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || N > kMaxColumns) return MOE_ERR_UNSUPPORTED;
  // one expert's codes are addressed with 31-bit byte offsets, tiles with 24 bits
  if (static_cast<int64_t>(N) * (K / 2) >= (static_cast<int64_t>(1) << 31)) return MOE_ERR_UNSUPPORTED;
  if (rows > (1 << 27)) return MOE_ERR_UNSUPPORTED;
  const int64_t tiles = (rows / 16 + (E < rows ? E : rows)) * ((N + 63) / 64);
  if (tiles >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_mxfp4_scale_bytes(int32_t K) {
  return K > 0 && K % kGroup == 0 && K <= kMaxK ? mx_scale_bytes(K) : 0;
}

int moe_mxfp4_quantize(const void* x, int32_t dtype, int64_t rows, int32_t K, int64_t x_stride,
                       int32_t* codes, uint8_t* scales, void* stream) {
  if (int st = check_mx(rows, K)) return st;
  if (int st = check_matrix(rows, K, x_stride, dtype)) return st;
  if (rows == 0) return MOE_OK;
  if (!ok_typed(x, dtype) || !ok_ptr(codes) || !ok_ptr(scales)) return MOE_ERR_INVALID_ARG;
  launch_mx_quantize(x, dtype, rows, K, x_stride, codes, scales, nullptr, 0, 0,
                     static_cast<hipStream_t>(stream));
  return check_launch();
}

int moe_mxfp4_dequantize(const int32_t* codes, const uint8_t* scales, int64_t rows, int32_t K,
                         void* x, int32_t dtype, int64_t x_stride, void* stream) {
  if (int st = check_mx(rows, K)) return st;
  if (int st = check_matrix(rows, K, x_stride, dtype)) return st;
  if (rows == 0) return MOE_OK;
  if (!ok_typed(x, dtype) || !ok_ptr(codes) || !ok_ptr(scales)) return MOE_ERR_INVALID_ARG;
  launch_mx_dequantize(codes, scales, rows, K, x, dtype, x_stride,
                       static_cast<hipStream_t>(stream));
  return check_launch();
}

int moe_mxfp4_grouped_gemm(const int32_t* a_codes, const uint8_t* a_scales, int64_t a_rows,
                           const int32_t* row_slots, int32_t top_k, int64_t rows,
                           const int32_t* expert_offsets, int32_t E, const int32_t* w_codes,
                           const uint8_t* w_scales, int32_t N, int32_t K, void* out,
                           int32_t out_dtype, int64_t out_stride, void* stream) {
  if (int st = check_product(a_rows, rows, top_k, row_slots != nullptr, expert_offsets != nullptr,
                             E, N, K))
    return st;
  if (int st = check_matrix(rows, N, out_stride, out_dtype)) return st;
  if (rows == 0) return MOE_OK;
  if (!ok_ptr(a_codes) || !ok_ptr(a_scales) || !ok_ptr(w_codes) || !ok_ptr(w_scales) ||
      !aligned16(row_slots) || !aligned16(expert_offsets) || !ok_typed(out, out_dtype))
    return MOE_ERR_INVALID_ARG;
  MxGemmArgs a{};
  a.a_codes = reinterpret_cast<const uint8_t*>(a_codes);
  a.a_scales = a_scales;
  a.a_rows = a_rows;
  a.row_slots = row_slots;
  a.top_k = top_k;
  a.rows = static_cast<int>(rows);
  a.offsets = expert_offsets;
  a.E = E;
  a.w_codes = reinterpret_cast<const uint8_t*>(w_codes);
  a.w_scales = w_scales;
  a.N = N;
  a.K = K;
  a.out = out;
  a.out_dtype = out_dtype;
  a.out_ld = out_stride;
  launch_mx_gemm(a, static_cast<hipStream_t>(stream));
  return check_launch();
}

int moe_mxfp4_gate_up(const int32_t* a_codes, const uint8_t* a_scales, int64_t a_rows,
                      const int32_t* row_slots, int32_t top_k, int64_t rows,
                      const int32_t* expert_offsets, int32_t E, const int32_t* w13_codes,
                      const uint8_t* w13_scales, int32_t I, int32_t H, int32_t* act_codes,
                      uint8_t* act_scales, void* stream) {
  if (I <= 0 || I % kGroup) return MOE_ERR_INVALID_ARG;
  if (I > kMaxColumns / 2) return MOE_ERR_UNSUPPORTED;
  if (int st = check_product(a_rows, rows, top_k, row_slots != nullptr, expert_offsets != nullptr,
                             E, 2 * I, H))
    return st;
  if (rows == 0) return MOE_OK;
  if (!ok_ptr(a_codes) || !ok_ptr(a_scales) || !ok_ptr(w13_codes) || !ok_ptr(w13_scales) ||
      !aligned16(row_slots) || !aligned16(expert_offsets) || !ok_ptr(act_codes) ||
      !ok_ptr(act_scales))
    return MOE_ERR_INVALID_ARG;
  MxGemmArgs a{};
  a.a_codes = reinterpret_cast<const uint8_t*>(a_codes);
  a.a_scales = a_scales;
  a.a_rows = a_rows;
  a.row_slots = row_slots;
  a.top_k = top_k;
  a.rows = static_cast<int>(rows);
  a.offsets = expert_offsets;
  a.E = E;
  a.w_codes = reinterpret_cast<const uint8_t*>(w13_codes);
  a.w_scales = w13_scales;
  a.N = 2 * I;
  a.K = H;
  a.act_codes = reinterpret_cast<uint8_t*>(act_codes);
  a.act_scales = act_scales;
  launch_mx_gemm(a, static_cast<hipStream_t>(stream));
  return check_launch();
}

// ---- the permutation ------------------------------------------------------------
size_t moe_permute_masked_workspace_bytes(int64_t T, int32_t top_k, int32_t E) {
  if (check_slots(T, top_k) != MOE_OK || E < 1 || E > kMaxExperts) return 0;
  return permute_masked_workspace_bytes(T, top_k, E);
}

int moe_permute_masked(const int32_t* topk_ids, int64_t T, int32_t top_k, int32_t first_expert,
                       int32_t E, int32_t* expert_offsets, int32_t* sorted_slots,
                       int32_t* slot_rows, int32_t* active_experts, int32_t* num_active,
                       void* workspace, size_t workspace_bytes, void* stream) {
  if (int st = check_slots(T, top_k)) return st;
  if (E < 1 || first_expert < 0) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || first_expert > INT32_MAX - kMaxExperts) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!ok_ptr(topk_ids) || !ok_ptr(expert_offsets) || !ok_ptr(sorted_slots) ||
      !ok_ptr(slot_rows) || !ok_ptr(active_experts) || !ok_ptr(num_active))
    return MOE_ERR_INVALID_ARG;
  const size_t need = permute_masked_workspace_bytes(T, top_k, E);
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  if (need > 0 && !ok_ptr(workspace)) return MOE_ERR_INVALID_ARG;
  launch_permute_masked(topk_ids, static_cast<int>(T), top_k, first_expert, E, expert_offsets,
                        sorted_slots, slot_rows, active_experts, num_active, workspace,
                        static_cast<hipStream_t>(stream));
  return check_launch();
}

int moe_dispatch(const void* x, int32_t dtype, int64_t T, int32_t top_k, int32_t H,
                 int64_t x_stride, const int32_t* slot_rows, int64_t rows, void* x_sorted,
                 int64_t sorted_stride, void* stream) {
  if (int st = check_rows(T, top_k, H, rows)) return st;
  if (int st = check_matrix(T, H, x_stride, dtype)) return st;
  if (int st = check_matrix(rows, H, sorted_stride, dtype)) return st;
  if (T == 0 || rows == 0) return MOE_OK;
  if (!ok_typed(x, dtype) || !ok_ptr(slot_rows) || !ok_typed(x_sorted, dtype))
    return MOE_ERR_INVALID_ARG;
  launch_dispatch(x, dtype_bytes(dtype), static_cast<int>(T), top_k, H, x_stride, slot_rows,
                  x_sorted, sorted_stride, static_cast<int>(rows),
                  static_cast<hipStream_t>(stream));
  return check_launch();
}

int moe_dispatch_backward(const void* grad_sorted, int32_t dtype, int64_t T, int32_t top_k,
                          int32_t H, int64_t sorted_stride, const int32_t* slot_rows, int64_t rows,
                          void* grad_x, int64_t x_stride, void* stream) {
  if (int st = check_rows(T, top_k, H, rows)) return st;
  if (int st = check_matrix(rows, H, sorted_stride, dtype)) return st;
  if (int st = check_matrix(T, H, x_stride, dtype)) return st;
  if (T == 0) return MOE_OK;
  if ((rows > 0 && !ok_typed(grad_sorted, dtype)) || !ok_ptr(slot_rows) || !ok_typed(grad_x, dtype))
    return MOE_ERR_INVALID_ARG;
  launch_combine_typed(grad_sorted, dtype, static_cast<int>(T), top_k, H, sorted_stride, nullptr,
                       slot_rows, static_cast<int>(rows), grad_x, dtype, x_stride,
                       static_cast<hipStream_t>(stream));
  return check_launch();
}

int moe_combine_masked(const void* y_sorted, int32_t y_dtype, int64_t T, int32_t top_k, int32_t H,
                       int64_t y_stride, const float* topk_weights, const int32_t* slot_rows,
                       int64_t rows, void* out, int32_t out_dtype, int64_t out_stride,
                       void* stream) {
  if (int st = check_rows(T, top_k, H, rows)) return st;
  if (int st = check_matrix(rows, H, y_stride, y_dtype)) return st;
  if (int st = check_matrix(T, H, out_stride, out_dtype)) return st;
  if (T == 0) return MOE_OK;
  if ((rows > 0 && !ok_typed(y_sorted, y_dtype)) || !ok_ptr(topk_weights) || !ok_ptr(slot_rows) ||
      !ok_typed(out, out_dtype))
    return MOE_ERR_INVALID_ARG;
  launch_combine_typed(y_sorted, y_dtype, static_cast<int>(T), top_k, H, y_stride, topk_weights,
                       slot_rows, static_cast<int>(rows), out, out_dtype, out_stride,
                       static_cast<hipStream_t>(stream));
  return check_launch();
}

int moe_combine_backward(const void* grad_out, int32_t grad_dtype, int64_t grad_stride,
                         const void* y_sorted, int32_t y_dtype, int64_t y_stride,
                         const float* topk_weights, const int32_t* slot_rows, int64_t T,
                         int32_t top_k, int32_t H, int64_t rows, void* grad_y,
                         int64_t grad_y_stride, float* grad_weights, void* stream) {
  if (int st = check_rows(T, top_k, H, rows)) return st;
  if (int st = check_matrix(T, H, grad_stride, grad_dtype)) return st;
  if (int st = check_matrix(rows, H, y_stride, y_dtype)) return st;
  if (int st = check_matrix(rows, H, grad_y_stride, y_dtype)) return st;
  if (T == 0) return MOE_OK;
  if (!ok_typed(grad_out, grad_dtype) ||
      (rows > 0 && (!ok_typed(y_sorted, y_dtype) || !ok_typed(grad_y, y_dtype))) ||
      !ok_ptr(topk_weights) || !ok_ptr(slot_rows) || !ok_ptr(grad_weights))
    return MOE_ERR_INVALID_ARG;
  launch_combine_backward(grad_out, grad_dtype, grad_stride, y_sorted, y_dtype, y_stride,
                          topk_weights, slot_rows, static_cast<int>(T), top_k, H,
                          static_cast<int>(rows), grad_y, grad_y_stride, grad_weights,
                          static_cast<hipStream_t>(stream));
  return check_launch();
}

// ---- the layer on MXFP4 experts ---------------------------------------------------
struct MxLayerWs {
  int32_t *ids, *offsets, *sorted, *slot_rows, *active, *num_active;
  float* weights;
  void* perm;
  size_t perm_bytes;
  int32_t *x_codes, *act_codes;
  uint8_t *x_scales, *act_scales;
  float* y;
  size_t total;
};

static MxLayerWs mx_layer_ws(void* base, int64_t T, int32_t top_k, int32_t E, int32_t H, int32_t I) {
  const size_t S = static_cast<size_t>(T) * top_k;
  char* p = static_cast<char*>(base);
  size_t at = 0;
  auto take = [&](size_t n) {
    char* q = p ? p + at : nullptr;
    at += align256(n);
    return q;
  };
  MxLayerWs w;
  w.ids = reinterpret_cast<int32_t*>(take(4 * S));
  w.weights = reinterpret_cast<float*>(take(4 * S));
  w.offsets = reinterpret_cast<int32_t*>(take(4 * (static_cast<size_t>(E) + 1)));
  w.sorted = reinterpret_cast<int32_t*>(take(4 * S));
  w.slot_rows = reinterpret_cast<int32_t*>(take(4 * S));
  w.active = reinterpret_cast<int32_t*>(take(4 * static_cast<size_t>(E)));
  w.num_active = reinterpret_cast<int32_t*>(take(4));
  w.perm_bytes = permute_masked_workspace_bytes(T, top_k, E);
  w.perm = take(w.perm_bytes);
  w.x_codes = reinterpret_cast<int32_t*>(take(S * (H / 2)));
  w.x_scales = reinterpret_cast<uint8_t*>(take(S * mx_scale_bytes(H)));
  w.act_codes = reinterpret_cast<int32_t*>(take(S * (I / 2)));
  w.act_scales = reinterpret_cast<uint8_t*>(take(S * mx_scale_bytes(I)));
  w.y = reinterpret_cast<float*>(take(4 * S * static_cast<size_t>(H)));
  w.total = at;
  return w;
}

// Sizes the layer takes: those of its calls.
static int check_mx_layer(int64_t T, int32_t top_k, int32_t E, int32_t H, int32_t I) {
  if (int st = check_slots(T, top_k)) return st;
  if (E < 1 || top_k > E || H <= 0 || H % kGroup || I <= 0 || I % kGroup) return MOE_ERR_INVALID_ARG;
  if (E > kMaxExperts || H > kMaxColumns || I > kMaxColumns / 2) return MOE_ERR_UNSUPPORTED;
  const int64_t S = T * top_k;
  if (int st = check_product(S, S, 1, false, true, E, 2 * I, H)) return st;
  return check_product(S, S, 1, false, true, E, H, I);
}

size_t moe_mxfp4_layer_workspace_bytes(int64_t T, int32_t top_k, int32_t E, int32_t H, int32_t I) {
  if (check_mx_layer(T, top_k, E, H, I) != MOE_OK) return 0;
  return mx_layer_ws(nullptr, T, top_k, E, H, I).total;
}

int moe_mxfp4_layer_forward(const float* logits, const void* x, int32_t dtype, int64_t T, int32_t E,
                            int32_t top_k, const int32_t* w13_codes, const uint8_t* w13_scales,
                            const int32_t* w2_codes, const uint8_t* w2_scales, int32_t H, int32_t I,
                            void* out, void* workspace, size_t workspace_bytes, void* stream) {
  if (!dtype_ok(dtype)) return MOE_ERR_INVALID_ARG;
  if (int st = check_mx_layer(T, top_k, E, H, I)) return st;
  if (T == 0) return MOE_OK;
  if (!ok_ptr(logits) || !ok_ptr(x) || !ok_ptr(w13_codes) || !ok_ptr(w13_scales) ||
      !ok_ptr(w2_codes) || !ok_ptr(w2_scales) || !ok_ptr(out) || !ok_ptr(workspace))
    return MOE_ERR_INVALID_ARG;
  const MxLayerWs w = mx_layer_ws(workspace, T, top_k, E, H, I);
  if (workspace_bytes < w.total) return MOE_ERR_WORKSPACE;
  const int64_t S = T * top_k;
  if (mx_small_ok(T, top_k, E, H, I)) {
    MxSmallArgs a{};
    a.logits = logits;
    a.x = x;
    a.dtype = dtype;
    a.T = static_cast<int>(T);
    a.E = E;
    a.top_k = top_k;
    a.H = H;
    a.I = I;
    a.w13_codes = reinterpret_cast<const uint8_t*>(w13_codes);
    a.w13_scales = w13_scales;
    a.w2_codes = reinterpret_cast<const uint8_t*>(w2_codes);
    a.w2_scales = w2_scales;
    a.ids = w.ids;
    a.weights = w.weights;
    a.act_codes = reinterpret_cast<uint8_t*>(w.act_codes);
    a.act_scales = w.act_scales;
    a.out = out;
    launch_mx_small_layer(a, static_cast<hipStream_t>(stream));
    return check_launch();
  }
  // one launch for few tokens; otherwise the masked permutation, which drops
  // nothing here: moe_permute's result in one launch less
  if (T <= kPermBlockTokens) {
    if (int st = moe_route_permute(logits, T, E, top_k, w.ids, w.weights, w.offsets, w.sorted,
                                   w.slot_rows, w.active, w.num_active, nullptr, 0, stream))
      return st;
  } else {
    if (int st = moe_route(logits, T, E, top_k, w.ids, w.weights, stream)) return st;
    if (int st = moe_permute_masked(w.ids, T, top_k, 0, E, w.offsets, w.sorted, w.slot_rows,
                                    w.active, w.num_active, w.perm, w.perm_bytes, stream))
      return st;
  }
  // every token once, stored to its rows: the products then read rows in order
  launch_mx_quantize(x, dtype, T, H, H, w.x_codes, w.x_scales, w.slot_rows, top_k,
                     static_cast<int>(S), static_cast<hipStream_t>(stream));
  if (int st = moe_mxfp4_gate_up(w.x_codes, w.x_scales, S, nullptr, 1, S, w.offsets, E, w13_codes,
                                 w13_scales, I, H, w.act_codes, w.act_scales, stream))
    return st;
  if (int st = moe_mxfp4_grouped_gemm(w.act_codes, w.act_scales, S, nullptr, 1, S, w.offsets, E,
                                      w2_codes, w2_scales, H, I, w.y, MOE_F32, H, stream))
    return st;
  return moe_combine_masked(w.y, MOE_F32, T, top_k, H, H, w.weights, w.slot_rows, S, out, dtype, H,
                            stream);
}

}  // extern "C"
