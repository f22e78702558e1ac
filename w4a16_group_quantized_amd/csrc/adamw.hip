// One AdamW step over many tensors:
//   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
//   p = p (1 - lr wd) - (lr / c1) m / (sqrt(v) / sqrt(c2) + eps),   c = 1 - b^step
// with m and v in fp32, or in 8 bits per element and one fp32 scale per block of
// 128.  Bound by memory: each value is read once and written once.  105 million
// elements: fp32 parameters and gradients and a bf16 copy, 8-bit states 324 to 345 us
// (5.5 to 5.8 TB/s), fp32 states 570 (5.5); bf16 parameters and gradients, no copy, 415
// us with fp32 states (5.6) and 195 to 231 with 8-bit ones (4.6 to 5.4: the noise's three
// multiplications an element are as long as its 10 bytes).  30 tensors of 2560 elements, one launch: 5 us.
//
// 8-bit states.  A block's scale is its largest magnitude / 1.875.  m has a sign,
// 4 exponent and 3 mantissa bits, v, which is not negative, 5 and 3: code c stands
// for scale times the small float whose fp32 bits are c << 20, moved to the range
// [0, 1.875] by a power of two (a code under 8 is subnormal there as in fp32, so
// one formula takes all).  Back to a code: add 20 noise bits behind the 3 mantissa
// bits and cut.  That rounds up with the probability of the part cut off, so the
// mean of many steps follows the moments; to nearest, a step's change of
// (1 - b2) = 0.1% would never pass half of a code's 6% and v would stand still under
// a scale that does (300 steps: 35% too large; with one noise for all steps 34%).
// The noise is a mix of the element's number and the step's seed, so a step is a
// function of its arguments.  A positive v never becomes 0: next to an m that did
// not, it would divide by eps.
#include "train.h"
#include "typed.h"

#include <float.h>

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kPerThread = 8;
constexpr int kPerGroup = kThreads * kPerThread;
// What fits in the 4 KiB of a launch's arguments.
constexpr int kTensors = 40;
constexpr int64_t kMaxLaunchGroups = 1 << 23;

struct Batch {
  moe_adamw_tensor t[kTensors];
  int32_t first[kTensors];  // workgroup that begins the tensor
  int count;
};
static_assert(sizeof(Batch) + sizeof(AdamwScalars) <= 4096 - 16, "kernel arguments");

// 8 bytes of codes at any address; past the first n they read as zero and are not stored.
struct __attribute__((packed, aligned(1), may_alias)) Bytes8 { uint64_t d; };
__device__ __forceinline__ uint64_t load_codes(const uint8_t* p, int n) {
  if (n >= 8) return reinterpret_cast<const Bytes8*>(p)->d;
  uint64_t d = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) d |= i < n ? static_cast<uint64_t>(p[i]) << (8 * i) : 0;
  return d;
}
__device__ __forceinline__ void store_codes(uint8_t* p, int n, uint64_t d) {
  if (n >= 8) {
    reinterpret_cast<Bytes8*>(p)->d = d;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) p[i] = static_cast<uint8_t>(d >> (8 * i));
}

__device__ __forceinline__ void load_any(const void* p, int dtype, int64_t at, int n,
                                         float (&v)[8]) {
  if (dtype == MOE_F32)
    load8<F32>(static_cast<const uint32_t*>(p) + at, n, v);
  else if (dtype == MOE_F16)
    load8<F16>(static_cast<const uint16_t*>(p) + at, n, v);
  else
    load8<BF16>(static_cast<const uint16_t*>(p) + at, n, v);
}
__device__ __forceinline__ void store_any(void* p, int dtype, int64_t at, int n,
                                          const float (&v)[8]) {
  if (dtype == MOE_F32)
    store8<F32>(static_cast<uint32_t*>(p) + at, n, v);
  else if (dtype == MOE_F16)
    store8<F16>(static_cast<uint16_t*>(p) + at, n, v);
  else
    store8<BF16>(static_cast<uint16_t*>(p) + at, n, v);
}

// Largest magnitude over the row of 16 lanes that holds a block, as its bits (those
// of a NaN are the largest).
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, static_cast<uint32_t>(
                    __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, false)));
}
__device__ __forceinline__ float block_max(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
  m = dpp_max<0xB1>(m);   // quad_perm [1,0,3,2]
  m = dpp_max<0x4E>(m);   // quad_perm [2,3,0,1]
  m = dpp_max<0x141>(m);  // row_half_mirror
  m = dpp_max<0x140>(m);  // row_mirror
  return __builtin_bit_cast(float, m);
}

constexpr float kPerTop = 1.f / 1.875f;  // 1.875: the largest code's value
constexpr float kLeast = 1.17549435e-38f;

template <bool SIGNED>
__device__ __forceinline__ float decode(uint32_t c, float scale) {
  const float small = __builtin_bit_cast(float, (SIGNED ? c & 127u : c) << 20);
  const float v = small * (SIGNED ? 0x1p112f : 0x1p96f) * scale;
  return SIGNED && (c & 128u) ? -v : v;
}

// The noise of 8 elements from number `at` on, 32 bits each.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x6A09E667u;
  x = (x ^ (x >> 15)) * 0xB7E15163u;
  return x ^ (x >> 16);
}

template <bool SIGNED>
__device__ __forceinline__ uint64_t encode(const float (&v)[8], const uint32_t (&noise)[8],
                                           float& scale) {
  // written out without fused steps: codes are a function of the values in fp32
#pragma clang fp contract(off)
  scale = block_max(v) * kPerTop;
  if (scale < kLeast) scale = 0.f;  // its reciprocal would not be finite
  const float inverse = scale == 0.f ? 0.f : 1.f / scale;
  uint64_t codes = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t bits = __builtin_bit_cast(uint32_t, v[i]);
    const float a = __builtin_bit_cast(float, bits & 0x7FFFFFFFu) * inverse;
    const float small = a * (SIGNED ? 0x1p-112f : 0x1p-96f);
    uint32_t c = (__builtin_bit_cast(uint32_t, small) + (noise[i] >> 12)) >> 20;
    c = min(c, SIGNED ? 127u : 255u);
    if (SIGNED)
      c |= (bits >> 31) << 7;
    else if (c == 0 && bits != 0)
      c = 1;
    codes |= static_cast<uint64_t>(c) << (8 * i);
  }
  return codes;
}

template <int BITS>
__global__ __launch_bounds__(kThreads) void adamw_kernel(Batch b, AdamwScalars s) {
  // the tensor that this workgroup belongs to
  int lo = 0, hi = b.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int>(blockIdx.x) >= b.first[mid])
      lo = mid;
    else
      hi = mid;
  }
  const moe_adamw_tensor& t = b.t[lo];
  const int64_t at = static_cast<int64_t>(static_cast<int>(blockIdx.x) - b.first[lo]) * kPerGroup +
                     threadIdx.x * kPerThread;
  const int n = static_cast<int>(min(max(t.n - at, int64_t{0}), int64_t{kPerThread}));
  const int64_t blk = at / kAdamwBlock;
  float p[8] = {}, g[8] = {}, m[8] = {}, v[8] = {};
  uint64_t mc = 0, vc = 0;
  float ms = 0.f, vs = 0.f;
  if (n > 0) {
    load_any(t.grad, t.grad_dtype, at, n, g);
    load_any(t.param, t.param_dtype, at, n, p);
    if constexpr (BITS == 32) {
      load8<F32>(static_cast<const uint32_t*>(t.m) + at, n, m);
      load8<F32>(static_cast<const uint32_t*>(t.v) + at, n, v);
    } else {
      mc = load_codes(static_cast<const uint8_t*>(t.m) + at, n);
      vc = load_codes(static_cast<const uint8_t*>(t.v) + at, n);
      ms = t.m_scales[blk];
      vs = t.v_scales[blk];
    }
  }
  if constexpr (BITS == 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      m[i] = i < n ? decode<true>(static_cast<uint32_t>(mc >> (8 * i)) & 255u, ms) : 0.f;
      v[i] = i < n ? decode<false>(static_cast<uint32_t>(vc >> (8 * i)) & 255u, vs) : 0.f;
    }
  }
  const float gs = s.grad_scale == nullptr ? 1.f : *s.grad_scale;
  {
#pragma clang fp contract(off)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float gi = i < n ? g[i] * gs : 0.f;
      m[i] = s.beta1 * m[i] + s.rest1 * gi;
      v[i] = s.beta2 * v[i] + s.rest2 * (gi * gi);
    }
  }
  float move[8];  // m / (sqrt(v) / sqrt(c2) + eps)
  if (s.small) {
    // The root's instruction takes v under 2^-126 for 0, and the reciprocal's an eps under it;
    // where eps is all there is, its reciprocal may also be past fp32's range while m is 0.
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool tiny = v[i] < 0x1p-96f;
      const float root =
          __builtin_amdgcn_sqrtf(v[i] * (tiny ? 0x1p64f : 1.f)) * (tiny ? 0x1p-32f : 1.f);
      const float over = fmaf(root, s.root, s.eps), up = over < 0x1p-64f ? 0x1p64f : 1.f;
      move[i] = m[i] * up * __builtin_amdgcn_rcpf(over * up);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      move[i] = m[i] * __builtin_amdgcn_rcpf(fmaf(__builtin_amdgcn_sqrtf(v[i]), s.root, s.eps));
  }
  // Both parts of the change are summed and p is rounded once: as a factor, 1 - lr wd is held in
  // steps of 2^-24, and a decay of a few of them would be off by as much of it (1e-7: 19 %).  An
  // infinity stays one: its decay is a finite number.
#pragma unroll
  for (int i = 0; i < 8; ++i)
    p[i] -= fmaf(s.size, move[i], s.decay * __builtin_amdgcn_fmed3f(p[i], -FLT_MAX, FLT_MAX));
  if constexpr (BITS == 8) {
    uint32_t noise[8], more[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint64_t e = at + i;
      noise[i] = mix(static_cast<uint32_t>(e) +
                     (s.seed + static_cast<uint32_t>(e >> 32)) * 0x9E3779B9u);
      more[i] = noise[i] * 0x9E3779B1u;
    }
    mc = encode<true>(m, noise, ms);
    vc = encode<false>(v, more, vs);
  }
  if (n <= 0) return;
  store_any(t.param, t.param_dtype, at, n, p);
  if (t.copy != nullptr) store_any(t.copy, t.copy_dtype, at, n, p);
  if constexpr (BITS == 32) {
    store8<F32>(static_cast<uint32_t*>(t.m) + at, n, m);
    store8<F32>(static_cast<uint32_t*>(t.v) + at, n, v);
  } else {
    store_codes(static_cast<uint8_t*>(t.m) + at, n, mc);
    store_codes(static_cast<uint8_t*>(t.v) + at, n, vc);
    if ((threadIdx.x & 15) == 0) {
      t.m_scales[blk] = ms;
      t.v_scales[blk] = vs;
    }
  }
}

}  // namespace

// As many launches as the tensors take: each holds its tensors' addresses in its
// arguments, so nothing is copied to the device beside them.
void launch_adamw(const moe_adamw_tensor* tensors, int count, int state_bits,
                  const AdamwScalars& s, hipStream_t stream) {
  Batch b;
  for (int i = 0; i < count;) {
    int64_t groups = 0;
    b.count = 0;
    for (; i < count && b.count < kTensors; ++i) {
      const int64_t mine = (tensors[i].n + kPerGroup - 1) / kPerGroup;
      if (mine == 0) continue;
      if (b.count > 0 && groups + mine > kMaxLaunchGroups) break;
      b.t[b.count] = tensors[i];
      b.first[b.count++] = static_cast<int32_t>(groups);
      groups += mine;
    }
    if (b.count == 0) continue;
    const dim3 grid(static_cast<unsigned>(groups));
    if (state_bits == 32)
      hipLaunchKernelGGL(adamw_kernel<32>, grid, dim3(kThreads), 0, stream, b, s);
    else
      hipLaunchKernelGGL(adamw_kernel<8>, grid, dim3(kThreads), 0, stream, b, s);
  }
}

}  // namespace moe
