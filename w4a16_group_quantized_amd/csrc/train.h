// Declarations of the training operators shared by their HIP translation units
// and the ABI layer (internal; not part of the public ABI).
#pragma once

#include "common.h"

namespace moe {

// The three products of rows grouped by expert, all C[i, j] = sum_q X[i, q] Y[j, q]
// in fp32 over fp16 or bf16 operands:
//   kOut      out[r, n]       rows of a       x W[e, n, :]      over k
//   kRows     grad_a[r, k]    rows of grad    x W[e, :, k]      over n
//   kWeights  grad_w[e, n, k] columns of grad x columns of a    over the expert's rows
enum class Product { kOut, kRows, kWeights };

// Division of 0 <= n < 2^31 by a number known at the launch: with 2^(c-1) < d <= 2^c and
// mul = ceil(2^(31+c) / d) < 2^32, n mul exceeds n 2^(31+c) / d by less than n d / d < 2^31
// <= 2^(31+c) / d, so its part above 2^(31+c) is n / d cut to an integer.
struct Divisor {
  uint32_t mul, shift;  // mul == 0: by 1
  Divisor() = default;
  explicit Divisor(uint32_t d) : mul(0), shift(0) {
    uint32_t c = 0;
    while ((1u << c) < d) ++c;
    if (c == 0) return;
    mul = static_cast<uint32_t>(((static_cast<uint64_t>(1) << (31 + c)) + d - 1) / d);
    shift = c - 1;
  }
  __host__ __device__ uint32_t operator()(uint32_t n) const {
    return mul == 0 ? n : static_cast<uint32_t>((static_cast<uint64_t>(n) * mul) >> 32) >> shift;
  }
};

struct GroupedArgs {
  const uint16_t* x;  // a (kOut) or grad: [rows, ...], row stride x_ld
  int64_t x_ld;
  const uint16_t* y;  // W [E, N, K], or a [rows, K] with row stride y_ld (kWeights)
  int64_t y_ld;
  int dtype;          // of x and y: MOE_F16 or MOE_BF16
  const int* offsets; // [E + 1], or null with E == 1
  int rows, E, N, K;
  void* out;
  int out_dtype;
  int64_t out_ld;     // kOut, kRows
  int accumulate;     // kWeights: added to what out holds
  float* partial;     // kWeights: workspace of grouped_workspace_bytes
  // set at the launch
  int row_tiles, col_tiles;  // row_tiles: of an expert, kWeights only
  int parts;                 // kWeights: shares of an expert's rows, each a sum of its own
  Divisor by_expert, by_group, by_parts;
};
size_t grouped_workspace_bytes(int64_t rows, int E, int N, int K);
// kWeights in parts (grouped_weights.hip): the arguments of the parts' own sums in the
// workspace, and the launch that adds them.
GroupedArgs grouped_part_sums(const GroupedArgs& a);
void launch_add_parts(const GroupedArgs& a, int parts, hipStream_t stream);
// With tiles of 16-byte loads (grouped_out.hip, grouped_rows.hip, grouped_weights.hip).
void launch_grouped_out(const GroupedArgs& a, hipStream_t stream);
void launch_grouped_rows(const GroupedArgs& a, hipStream_t stream);
void launch_grouped_weights(const GroupedArgs& a, hipStream_t stream);
void launch_grouped(Product p, const GroupedArgs& a, hipStream_t stream);

// act = SiLU(gate) * up of h = [gate | up], rows [offsets[0], offsets[E]) or all.
struct ActArgs {
  const void* grad;   // backward only
  int64_t grad_ld;
  const void* h;
  int64_t h_ld;
  int dtype;
  int rows, I;
  const int* offsets;
  int E;
  void* out;          // act, or the gradient of h
  int64_t out_ld;
};
void launch_silu_mul(const ActArgs& a, bool backward, hipStream_t stream);

void launch_route_backward(const int* ids, const float* weights, const float* grad, int T, int E,
                           int top_k, void* out, int out_dtype, hipStream_t stream);

struct AdamwScalars {
  float beta1, rest1, beta2, rest2;  // rest = 1 - beta
  float decay, size, root, eps;      // lr wd, lr / c1, 1 / sqrt(c2)
  const float* grad_scale;           // device, or null: 1
  uint32_t seed;
  int small;                         // eps does not cover the root of v = 2^-126, or is under it
};
void launch_adamw(const moe_adamw_tensor* tensors, int count, int state_bits,
                  const AdamwScalars& s, hipStream_t stream);
constexpr int kAdamwBlock = MOE_ADAMW_BLOCK;

}  // namespace moe
