// Device helpers for the operators whose tensors may be fp32, fp16 or bf16
// (internal; not part of the public ABI): element types, loads and
// stores of 8 elements as fp32, and host-side dispatch over the types.
#pragma once

#include "common.h"

namespace moe {

struct F32 { using bits = uint32_t; };
struct F16 { using bits = uint16_t; };
struct BF16 { using bits = uint16_t; };

template <typename T>
constexpr int kBytes = sizeof(typename T::bits);

__device__ __forceinline__ float to_float(F32, uint32_t b) { return __builtin_bit_cast(float, b); }
__device__ __forceinline__ float to_float(F16, uint16_t b) { return half_bits_to_float(b); }
__device__ __forceinline__ float to_float(BF16, uint16_t b) {
  return __builtin_bit_cast(float, static_cast<uint32_t>(b) << 16);
}

// Every conversion to 16 bits rounds to nearest even, once, at the store.
__device__ __forceinline__ uint32_t from_float(F32, float f) { return __builtin_bit_cast(uint32_t, f); }
__device__ __forceinline__ uint16_t from_float(F16, float f) { return float_to_half_bits(f); }
__device__ __forceinline__ uint16_t from_float(BF16, float f) {
  return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}

// Up to 8 consecutive elements as fp32; past the first n they read as zero and
// are not stored.  Addresses need only the element's own alignment: the
// hardware takes 16-byte accesses at any address, and rows of odd length or
// stride would otherwise fall back to one element per access.
typedef uint32_t dwords4 __attribute__((ext_vector_type(4)));
struct __attribute__((packed, aligned(2), may_alias)) Unaligned16 { dwords4 d; };

__device__ __forceinline__ dwords4 load16(const void* p) {
  return reinterpret_cast<const Unaligned16*>(p)->d;
}
// Nontemporal, against plain stores: 4096 tokens x 10 x 2560 bf16, dispatch 38 us
// against 41, combine 43 against 46, combine backward 82 against 84; 10240 rows of
// the down product 117 against 122.  Rows of 8 tokens take the same time either way
// (4.0 us); the layer of 8 tokens, whose next launch reads the fp32 rows back, is
// 2 us slower for it (78 against 76 us), that of 1024 tokens is not (357 and 358).
__device__ __forceinline__ void store16(void* p, dwords4 d) {
  __builtin_nontemporal_store(d, &reinterpret_cast<Unaligned16*>(p)->d);
}

template <typename T>
__device__ __forceinline__ void load8(const typename T::bits* p, int n, float (&v)[8]) {
  if (n >= 8) {
    constexpr int E = 16 / kBytes<T>;
#pragma unroll
    for (int i = 0; i < 8; i += E) {
      const dwords4 d = load16(p + i);
#pragma unroll
      for (int j = 0; j < E; ++j) {
        if constexpr (kBytes<T> == 4)
          v[i + j] = __builtin_bit_cast(float, static_cast<uint32_t>(d[j]));
        else
          v[i + j] = to_float(T{}, static_cast<uint16_t>(d[j / 2] >> (16 * (j & 1))));
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? to_float(T{}, p[i]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store8(typename T::bits* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    constexpr int E = 16 / kBytes<T>;
#pragma unroll
    for (int i = 0; i < 8; i += E) {
      dwords4 d;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (kBytes<T> == 4)
          d[j] = __builtin_bit_cast(uint32_t, v[i + j]);
        else
          d[j] = static_cast<uint32_t>(from_float(T{}, v[i + 2 * j])) |
                 (static_cast<uint32_t>(from_float(T{}, v[i + 2 * j + 1])) << 16);
      }
      store16(p + i, d);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = from_float(T{}, v[i]);
  }
}

// ---- host side ---------------------------------------------------------------
inline int dtype_bytes(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
inline bool dtype_ok(int dtype) {
  return dtype == MOE_F32 || dtype == MOE_F16 || dtype == MOE_BF16;
}

// Calls f(F32{} / F16{} / BF16{}) for a valid dtype code.
template <typename F>
inline void with_dtype(int dtype, F&& f) {
  if (dtype == MOE_F32)
    f(F32{});
  else if (dtype == MOE_F16)
    f(F16{});
  else
    f(BF16{});
}

}  // namespace moe
