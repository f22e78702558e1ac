// MXFP4 quantisation and dequantisation.  A block is 32 consecutive values of
// a row.  With m = max |x| of the block:
//   e     = clamp(floor(log2 m) - 2, -127, 127)      (2: E2M1's largest exponent)
//   code  = nearest E2M1 value of x 2^-e, ties to even, at most 6 in size
//   scale = e + 127, one byte
// A zero block has e = -127; a block that holds an infinity or a NaN has scale
// byte 255, which stands for NaN, and zero codes.
//
// Both are bound by memory: one pass, 8 values (one code word) per lane, so
// loads and code stores of a wave are contiguous; the four lanes of a block
// meet by DPP inside their quad.  m is the largest bit pattern with the sign
// cleared, so an infinity or a NaN shows in the same maximum.  81920 x 2560
// bf16: 90 us there (5.9 TB/s), 85 us back (6.2 TB/s).
#include "mxfp4.h"
#include "mxfp4_tile.h"
#include "typed.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
// Code words per lane, their loads in flight together: 81920 x 2560 bf16 rows
// take 91 us with 2 (97 with 4, 99 with 1), and back 86 us with 4 (88 with 2).
constexpr int kQuantUnroll = 2;
constexpr int kDequantUnroll = 4;
constexpr int kMaxBlocks = 1 << 20;

// SCATTER: row t goes to rows slot_rows[t top_k + j] < out_rows, j < top_k,
// instead of row t (the rows of a token in expert order).
template <typename T, bool SCATTER>
__global__ __launch_bounds__(kThreads) void quantize_kernel(
    const typename T::bits* __restrict__ x, int64_t rows, int words, int64_t ld,
    uint32_t* __restrict__ codes, uint8_t* __restrict__ scales, int sbytes,
    const int* __restrict__ slot_rows, int top_k, int out_rows) {
  const int64_t total = rows * words;
  constexpr int kPerBlock = kThreads * kQuantUnroll;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kPerBlock; base < total;
       base += static_cast<int64_t>(gridDim.x) * kPerBlock) {
    const int64_t row0 = base / words;
    const uint32_t rem0 = static_cast<uint32_t>(base - row0 * words);
    float v[kQuantUnroll][8];
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) {
      const uint32_t off = rem0 + u * kThreads + threadIdx.x;
      const uint32_t r = off / static_cast<uint32_t>(words);
      const int64_t row = row0 + r;
      if (row < rows) {
        load8<T>(x + row * ld + 8 * static_cast<int64_t>(off - r * words), 8, v[u]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[u][i] = 0.f;
      }
    }
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) {
      const uint32_t off = rem0 + u * kThreads + threadIdx.x;
      const uint32_t r = off / static_cast<uint32_t>(words);
      const uint32_t c = off - r * words;
      const int64_t row = row0 + r;
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        m = max(m, abs_bits(v[u][i]));
      }
      m = quad_max<0xB1>(m);  // lanes 1 0 3 2
      m = quad_max<0x4E>(m);  // lanes 2 3 0 1
      const uint32_t byte = mx_scale_byte(m);
      const uint32_t q = mx_word(v[u], byte);
      if (row < rows) {
        auto put = [&](int64_t to) {
          codes[to * words + c] = q;
          if ((c & 3) == 0) store_scale(scales + to * sbytes, c >> 2, words >> 2, sbytes, byte);
        };
        if constexpr (SCATTER) {
          // eight places at a time: their loads are in flight together
          for (int j0 = 0; j0 < top_k; j0 += 8) {
            int to[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              to[j] = j0 + j < top_k ? slot_rows[row * top_k + j0 + j] : -1;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (static_cast<uint32_t>(to[j]) < static_cast<uint32_t>(out_rows)) put(to[j]);
          }
        } else {
          __builtin_nontemporal_store(q, codes + row * words + c);
          if ((c & 3) == 0) store_scale(scales + row * sbytes, c >> 2, words >> 2, sbytes, byte);
        }
      }
    }
  }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void dequantize_kernel(
    const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t rows, int words,
    int sbytes, typename T::bits* __restrict__ x, int64_t ld) {
  const int64_t total = rows * words;
  constexpr int kPerBlock = kThreads * kDequantUnroll;
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * kPerBlock; base < total;
       base += static_cast<int64_t>(gridDim.x) * kPerBlock) {
    const int64_t row0 = base / words;
    const uint32_t rem0 = static_cast<uint32_t>(base - row0 * words);
    uint32_t q[kDequantUnroll], s[kDequantUnroll];
#pragma unroll
    for (int u = 0; u < kDequantUnroll; ++u) {
      const uint32_t off = rem0 + u * kThreads + threadIdx.x;
      const uint32_t r = off / static_cast<uint32_t>(words);
      const uint32_t c = off - r * words;
      const int64_t row = row0 + r;
      q[u] = row < rows ? codes[row * words + c] : 0u;
      s[u] = row < rows ? scales[row * sbytes + (c >> 2)] : 0u;
    }
#pragma unroll
    for (int u = 0; u < kDequantUnroll; ++u) {
      const uint32_t off = rem0 + u * kThreads + threadIdx.x;
      const uint32_t r = off / static_cast<uint32_t>(words);
      const uint32_t c = off - r * words;
      const int64_t row = row0 + r;
      const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 0);
      const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 1);
      const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 2);
      const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[u], 1.f, 3);
      float v[8] = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
      const int e = static_cast<int>(s[u]) - 127;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        v[i] = s[u] == 255u ? __builtin_nanf("") : ldexpf(v[i], e);
      if (row < rows) store8<T>(x + row * ld + 8 * static_cast<int64_t>(c), 8, v);
    }
  }
}

int grid_for(int64_t rows, int words, int unroll) {
  const int64_t n = (rows * words + kThreads * unroll - 1) / (kThreads * unroll);
  return static_cast<int>(n < kMaxBlocks ? n : kMaxBlocks);
}

}  // namespace

void launch_mx_quantize(const void* x, int dtype, int64_t rows, int K, int64_t ld, int32_t* codes,
                        uint8_t* scales, const int* slot_rows, int top_k, int out_rows,
                        hipStream_t stream) {
  const int words = K / 8;
  const dim3 grid(grid_for(rows, words, kQuantUnroll));
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    const auto* p = static_cast<const typename T::bits*>(x);
    auto* q = reinterpret_cast<uint32_t*>(codes);
    if (slot_rows != nullptr)
      hipLaunchKernelGGL((quantize_kernel<T, true>), grid, dim3(kThreads), 0, stream, p, rows, words,
                         ld, q, scales, mx_scale_bytes(K), slot_rows, top_k, out_rows);
    else
      hipLaunchKernelGGL((quantize_kernel<T, false>), grid, dim3(kThreads), 0, stream, p, rows,
                         words, ld, q, scales, mx_scale_bytes(K), slot_rows, top_k, out_rows);
  });
}

void launch_mx_dequantize(const int32_t* codes, const uint8_t* scales, int64_t rows, int K, void* x,
                          int dtype, int64_t ld, hipStream_t stream) {
  const int words = K / 8;
  const dim3 grid(grid_for(rows, words, kDequantUnroll));
  with_dtype(dtype, [&](auto t) {
    using T = decltype(t);
    auto* p = static_cast<typename T::bits*>(x);
    const auto* q = reinterpret_cast<const uint32_t*>(codes);
    hipLaunchKernelGGL(dequantize_kernel<T>, grid, dim3(kThreads), 0, stream, q, scales,
                       rows, words, mx_scale_bytes(K), p, ld);
  });
}

}  // namespace moe
