// Device helpers of the MXFP4 products: scaled matrix operands, buffer loads
// and the quantising epilogue.
#pragma once

#include "mxfp4.h"
#include "tiles.h"
#include "typed.h"

namespace moe {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kFp4 = 4;                          // operand format code: E2M1

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0), bytes,
                                           kRawBuffer);
}
__device__ __forceinline__ dwords4 buffer_load16(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(dwords4, __builtin_amdgcn_raw_buffer_load_b128(r, static_cast<int>(at), 0, 0));
}
__device__ __forceinline__ uint32_t buffer_load4(__amdgpu_buffer_rsrc_t r, uint32_t at) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, static_cast<int>(at), 0, 0);
}
// 16 bytes at a 4-byte aligned address.
__device__ __forceinline__ dwords4 load_words4(const void* p) {
  struct __attribute__((packed, aligned(4), may_alias)) Words { dwords4 d; };
  return static_cast<const Words*>(p)->d;
}

// The instruction takes eight registers for its widest formats and reads the
// first four for 4-bit codes.
__device__ __forceinline__ i32x8 operand(dwords4 d) {
  return __builtin_bit_cast(i32x8, __builtin_shufflevector(d, d, 0, 1, 2, 3, -1, -1, -1, -1));
}

// Row of A that output row r takes (-1: none).
__device__ __forceinline__ int64_t a_row(const MxGemmArgs& p, int r) {
  if (p.row_slots == nullptr) return r;
  const int s = p.row_slots[r];
  if (s < 0) return -1;
  const int t = s / p.top_k;
  return t < p.a_rows ? t : -1;
}

// ---- the quantising epilogue ---------------------------------------------------
// gate / (1 + e^-gate) * up in a dozen instructions (the library's exponential
// and division made the epilogue the longest part of the gate/up product).
// With x = -gate, e^x = 2^t (1 + r ln 2), t = x log2(e) rounded and r what that
// rounding left, so the exponential is good to 2 units in the last place while it
// is a normal number, the hardware's reciprocal to 1 down to 2^-126.  x is held in
// [-128, 128], outside which e^x is 0 or past fp32 anyway: t of a finite gate past
// 2.3e38 would be infinite and r with it, and 0 times r a NaN.  Below a gate of
// -87.3 the reciprocal is under 2^-126 and counts as 0: what is lost is under
// 2^-126 |gate up|.  A NaN gate stays NaN through the last product.
__device__ __forceinline__ float silu_mul(float gate, float up) {
  constexpr float kLog2e = 1.44269504f, kLog2eRest = 1.92596299e-8f, kLn2 = 0.693147181f;
  const float x = __builtin_amdgcn_fmed3f(-gate, -128.f, 128.f);
  const float t = x * kLog2e;
  const float r = fmaf(x, kLog2eRest, fmaf(x, kLog2e, -t));
  const float e = __builtin_amdgcn_exp2f(t) * fmaf(r, kLn2, 1.f);
  return gate * __builtin_amdgcn_rcpf(1.f + e) * up;
}
__device__ __forceinline__ uint32_t abs_bits(float v) {
  return __builtin_bit_cast(uint32_t, v) & 0x7FFFFFFFu;
}
// The scale byte of a block whose largest magnitude has bits m (255: it holds
// an infinity or a NaN).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t m) {
  const uint32_t field = m >> 23;
  return field == 255 ? 255u : (field > 2 ? field - 2 : 0u);
}
// Codes of two values in the low byte (zero for a NaN block).
__device__ __forceinline__ uint32_t mx_pair(float a, float b, uint32_t byte) {
  const float inv = __builtin_bit_cast(float, (254u - byte) << 23);
  if (byte == 255) return 0;
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, a * inv, b * inv, 1.f, 0) & 0xFFu;
}
// All eight codes of a word (v as loaded, byte their block's).
__device__ __forceinline__ uint32_t mx_word(const float (&v)[8], uint32_t byte) {
  // 2^-e; an exact product unless it is far below the smallest code
  const float inv = __builtin_bit_cast(float, (254u - byte) << 23);
  uint32_t q = 0;
  if (byte != 255) {
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[0] * inv, v[1] * inv, 1.f, 0);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[2] * inv, v[3] * inv, 1.f, 1);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[4] * inv, v[5] * inv, 1.f, 2);
    q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, v[6] * inv, v[7] * inv, 1.f, 3);
  }
  return q;
}
// Maximum with a neighbour in the quad (CTRL: quad permutation).
template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  const uint32_t o = __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);
  return v > o ? v : o;
}
// Block `blk`'s scale of a row of `blocks`; the last one also sets the row's
// padding, which stands for 1.
__device__ __forceinline__ void store_scale(uint8_t* row, int blk, int blocks, int sbytes,
                                            uint32_t byte) {
  row[blk] = static_cast<uint8_t>(byte);
  if (blk + 1 == blocks)
    for (int p = blocks; p < sbytes; ++p) row[p] = 127;
}

// SiLU(gate) * up of a tile of 16 tokens x 32 columns of I, stored as MXFP4 (the
// 32 columns are one block): of each four waves, 0 and 1 hold the gate's two
// halves in acc, 2 and 3 the up's, lane (col, g) columns 4 g ... + 3 of token col;
// PARTS fours of waves hold parts of the sums.  `h` is LDS of the workgroup.
template <int PARTS>
__device__ __forceinline__ void gate_up_epilogue(f32x4 acc, float (&h)[4 * PARTS][16][17], int wave,
                                                 int I, int nt, int r0, int rows,
                                                 uint8_t* act_codes, uint8_t* act_scales) {
  const int col = threadIdx.x & 15, g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) h[wave][col][4 * g + i] = acc[i];
  __syncthreads();
  if (threadIdx.x >= 256) return;
  // 16 threads per token, two neighbouring columns each
  const int t = threadIdx.x >> 4, c = (threadIdx.x & 15) * 2;
  float a[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    float gate = 0.f, up = 0.f;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      gate += h[4 * p + (c >> 4)][t][(c & 15) + q];
      up += h[4 * p + 2 + (c >> 4)][t][(c & 15) + q];
    }
    a[q] = silu_mul(gate, up);
  }
  uint32_t m = max(abs_bits(a[0]), abs_bits(a[1]));
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) m = max(m, static_cast<uint32_t>(__shfl_xor(m, d, 16)));
  const uint32_t byte = mx_scale_byte(m);
  uint32_t q = mx_pair(a[0], a[1], byte);
  q |= __shfl_xor(q, 1, 16) << 8;   // valid in even threads
  q |= __shfl_xor(q, 2, 16) << 16;  // valid in every fourth
  if (t < rows) {
    const int64_t row = r0 + t;
    const int sb = mx_scale_bytes(I);
    if ((threadIdx.x & 3) == 0)
      *reinterpret_cast<uint32_t*>(act_codes + row * (I / 2) + nt * 16 + c / 2) = q;
    if ((threadIdx.x & 15) == 0) store_scale(act_scales + row * sb, nt, I / 32, sb, byte);
  }
}

}  // namespace moe
