// Internal declarations of the MXFP4 operators and of the typed token
// permutation (launchers; each enqueues on `stream`, arguments checked by the
// ABI layer).
#pragma once

#include "common.h"

namespace moe {

// Bytes of one row's block scales: one per 32 values, rows padded to whole
// 32-bit words so that a lane takes the scales of 128 values with one load.
__host__ __device__ constexpr int mx_scale_bytes(int K) { return 4 * ((K + 127) / 128); }

// slot_rows (nullable): row t goes to rows slot_rows[t top_k + j] < out_rows.
void launch_mx_quantize(const void* x, int dtype, int64_t rows, int K, int64_t ld, int32_t* codes,
                        uint8_t* scales, const int* slot_rows, int top_k, int out_rows,
                        hipStream_t stream);
void launch_mx_dequantize(const int32_t* codes, const uint8_t* scales, int64_t rows, int K, void* x,
                          int dtype, int64_t ld, hipStream_t stream);

// A grouped product over expert segments; exactly one of out / act_codes is
// set (act_codes: N = 2I rows of gate and up, SiLU(gate)*up stored as MXFP4).
struct MxGemmArgs {
  const uint8_t* a_codes;    // [a_rows, K / 2]
  const uint8_t* a_scales;   // [a_rows, mx_scale_bytes(K)]
  int64_t a_rows;
  const int* row_slots;      // nullable: A row of output row r is row_slots[r] / top_k
  int top_k;
  int rows;                  // output rows
  const int* offsets;        // [E + 1]; null with E == 1: all rows
  int E;
  const uint8_t* w_codes;    // [E, N, K / 2]
  const uint8_t* w_scales;   // [E, N, mx_scale_bytes(K)]
  int N, K;
  void* out;
  int out_dtype;
  int64_t out_ld;
  uint8_t* act_codes;        // [rows, I / 2]
  uint8_t* act_scales;       // [rows, mx_scale_bytes(I)]
};
void launch_mx_gemm(const MxGemmArgs& a, hipStream_t stream);

// The whole layer for a few tokens, in two launches (mxfp4_small.hip).
constexpr int kMxSmallTokens = 6;
constexpr int kMxSmallHidden = 16384;  // 6 tokens of quantised x in LDS: 51 KB
struct MxSmallArgs {
  const float* logits;
  const void* x;
  int dtype;                 // of x and out
  int T, E, top_k, H, I;
  const uint8_t *w13_codes, *w13_scales, *w2_codes, *w2_scales;
  int* ids;                  // [T, top_k], written by the first launch
  float* weights;
  uint8_t *act_codes, *act_scales;
  void* out;
};
bool mx_small_ok(int64_t T, int top_k, int E, int H, int I);
void launch_mx_small_layer(const MxSmallArgs& p, hipStream_t stream);

size_t permute_masked_workspace_bytes(int64_t T, int top_k, int E);
void launch_permute_masked(const int* ids, int T, int top_k, int first, int E, int* offsets,
                           int* sorted_slots, int* slot_rows, int* active, int* num_active,
                           void* workspace, hipStream_t stream);

// Row movement; `rows` bounds every row index (others are skipped).
void launch_dispatch(const void* x, int bytes, int T, int top_k, int H, int64_t x_ld,
                     const int* slot_rows, void* out, int64_t out_ld, int rows,
                     hipStream_t stream);
void launch_combine_typed(const void* y, int y_dtype, int T, int top_k, int H, int64_t y_ld,
                          const float* weights, const int* slot_rows, int rows, void* out,
                          int out_dtype, int64_t out_ld, hipStream_t stream);
void launch_combine_backward(const void* grad, int grad_dtype, int64_t grad_ld, const void* y,
                             int y_dtype, int64_t y_ld, const float* weights,
                             const int* slot_rows, int T, int top_k, int H, int rows,
                             void* grad_y, int64_t grad_y_ld, float* grad_weights,
                             hipStream_t stream);

}  // namespace moe
