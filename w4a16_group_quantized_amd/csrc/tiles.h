// Device helpers of the grouped products: the tile search over expert segments,
// loads from memory straight to LDS with their waits, and rounded stores
// (internal; not part of the public ABI).
#pragma once

#include "typed.h"

namespace moe {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr uint32_t kOutOfRange = 0x80000000u;  // past every descriptor's range (< 2^31 bytes)
constexpr int kRawBuffer = 0x00020000;         // descriptor word 3: raw access on gfx9

// The experts' rows cut into tiles of `size`, experts ascending; an expert's
// last tile may be short.  The whole wave counts: lane l the tiles of experts
// [l per, (l + 1) per), then a scan over the lanes.  Offsets are held inside
// [0, rows]: an entry outside does not lead out of the tensors.  That they
// ascend is the caller's to keep.
constexpr int kHeld = 8;  // experts per lane whose offsets stay in registers

struct Tiles {
  const int* offsets;
  int E, rows, size;
  int per;             // experts per lane
  int inc, sum;        // this lane's share: tiles up to its end, tiles in it
  int o[kHeld + 1];    // its first offsets (all of them when per <= kHeld)
  int total;
};

__device__ __forceinline__ int tile_count(int a, int b, int size) {
  return (max(b - a, 0) + size - 1) / size;
}

// Inclusive sum over the lanes up to this one.
__device__ __forceinline__ int wave_scan(int v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d, 64);
    if (lane >= d) v += o;
  }
  return v;
}

__device__ __forceinline__ Tiles count_tiles(const int* __restrict__ offsets, int E, int rows,
                                             int size) {
  Tiles t{offsets, E, rows, size, (E + 63) >> 6, 0, 0, {}, 0};
  if (offsets == nullptr) {
    t.total = (rows + size - 1) / size;
    return t;
  }
  const int lane = threadIdx.x & 63;
  auto share = [&](int i0, int (&o)[kHeld + 1]) {
#pragma unroll
    for (int i = 0; i <= kHeld; ++i)
      o[i] = min(max(offsets[min(lane * t.per + min(i0 + i, t.per), E)], 0), rows);
#pragma unroll
    for (int i = 0; i < kHeld; ++i) t.sum += tile_count(o[i], o[i + 1], size);
  };
  share(0, t.o);
  for (int i0 = kHeld; i0 < t.per; i0 += kHeld) {
    int o[kHeld + 1];
    share(i0, o);
  }
  t.inc = wave_scan(t.sum);
  t.total = __builtin_amdgcn_readlane(t.inc, 63);
  return t;
}

// The counts kept in LDS between searches (they would hold a dozen registers
// through a kernel's main loop): every wave writes the same values.
struct TileTable {
  int inc[64], sum[64], o[kHeld + 1][64];
};

__device__ __forceinline__ int keep_tiles(const Tiles& t, TileTable& table) {
  if (t.offsets != nullptr) {
    const int lane = threadIdx.x & 63;
    table.inc[lane] = t.inc;
    table.sum[lane] = t.sum;
#pragma unroll
    for (int i = 0; i <= kHeld; ++i) table.o[i][lane] = t.o[i];
  }
  return t.total;
}

__device__ __forceinline__ Tiles kept_tiles(const TileTable& table, const int* offsets, int E,
                                            int rows, int size, int total) {
  Tiles t{offsets, E, rows, size, (E + 63) >> 6, 0, 0, {}, total};
  if (offsets != nullptr) {
    const int lane = threadIdx.x & 63;
    t.inc = table.inc[lane];
    t.sum = table.sum[lane];
#pragma unroll
    for (int i = 0; i <= kHeld; ++i) t.o[i] = table.o[i][lane];
  }
  return t;
}

// Tile mt's expert and rows [r0, r1); false behind the last tile.
__device__ __forceinline__ bool find_tile(const Tiles& t, int mt, int& e, int& r0, int& r1) {
  if (mt >= t.total) return false;
  if (t.offsets == nullptr) {
    e = 0;
    r0 = mt * t.size;
    r1 = min(t.rows, r0 + t.size);
    return true;
  }
  const int owner = __builtin_ctzll(__ballot(t.inc > mt));
  int at = __builtin_amdgcn_readlane(t.inc - t.sum, owner);  // tiles before the owner's experts
  if (t.per <= kHeld) {
    int b = __builtin_amdgcn_readlane(t.o[0], owner);
    bool found = false;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int a = b;
      b = __builtin_amdgcn_readlane(t.o[i + 1], owner);
      const int n = tile_count(a, b, t.size);
      if (!found && mt < at + n) {
        found = true;
        e = owner * t.per + i;
        r0 = a + (mt - at) * t.size;
        r1 = min(b, r0 + t.size);
      }
      at += n;
    }
    return found;
  }
  // more experts per lane: the lanes share out the owner's
  const int lane = threadIdx.x & 63;
  const int mine = min(owner * t.per + min(lane, t.per), t.E);
  const int a = min(max(t.offsets[mine], 0), t.rows);
  const int b = min(max(t.offsets[min(mine + 1, t.E)], 0), t.rows);
  const int n = lane < t.per ? tile_count(a, b, t.size) : 0;
  const int inc = wave_scan(n);
  const int who = __builtin_ctzll(__ballot(at + inc > mt));
  at += __builtin_amdgcn_readlane(inc - n, who);
  e = owner * t.per + who;
  r0 = __builtin_amdgcn_readlane(a, who) + (mt - at) * t.size;
  r1 = min(__builtin_amdgcn_readlane(b, who), r0 + t.size);
  return true;
}

typedef uint32_t dwords2 __attribute__((ext_vector_type(2)));

// Two values rounded to nearest even, in one word, low half first: one instruction for
// both.
__device__ __forceinline__ uint32_t pack2(F16, float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, h2_t));
}
__device__ __forceinline__ uint32_t pack2(BF16, float a, float b) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, b2_t));
}
// Four results of a 16-bit type, rounded, in two words.
template <typename T>
__device__ __forceinline__ dwords2 pack4(f32x4 v) {
  return dwords2{pack2(T{}, v[0], v[1]), pack2(T{}, v[2], v[3])};
}

template <typename T>
__device__ __forceinline__ void store4(typename T::bits* p, int n, f32x4 v) {
  if (n >= 4) {
    if constexpr (kBytes<T> == 4) {
      store16(p, __builtin_bit_cast(dwords4, v));
    } else {
      struct __attribute__((packed, aligned(2), may_alias)) Unaligned8 { dwords2 d; };
      reinterpret_cast<Unaligned8*>(p)->d = pack4<T>(v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = from_float(T{}, v[i]);
  }
}

// Loads from memory straight to LDS, 16 or 4 bytes per lane: from the lane's
// offset `at` to consecutive places from LDS address `lds` on.  Written out
// because the compiler, which does not see which stage a read of LDS meets,
// would wait for every load on its way before it; the waits are
// wait_loads_and_barrier's.  There is no result register that could be reused
// too early, and the LDS arrays' addresses are taken, so what the memory
// barriers of the waits cover includes them.
struct Descriptor {
  dwords4 d;
};

__device__ __forceinline__ Descriptor descriptor(const void* base, uint32_t bytes) {
  const uint64_t at = reinterpret_cast<uint64_t>(base);
  Descriptor r;
  r.d[0] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at));
  r.d[1] = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(at >> 32)) & 0xFFFFu;
  r.d[2] = __builtin_amdgcn_readfirstlane(bytes);
  r.d[3] = kRawBuffer;
  return r;
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(
      (__attribute__((address_space(3))) const void*)p));
}

__device__ __forceinline__ void load16_to_lds(const Descriptor& r, uint32_t lds, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds),
               "v"(at), "s"(r.d)
               : "m0");
}
__device__ __forceinline__ void load4_to_lds(const Descriptor& r, uint32_t lds, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds),
               "v"(at), "s"(r.d)
               : "m0");
}

template <int N>
__device__ __forceinline__ void wait_loads_and_barrier() {
  // all but the N newest loads done, LDS reads done, then the barrier; nothing
  // that touches memory moves across
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ void wait_lds_and_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);  // LDS only
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace moe
