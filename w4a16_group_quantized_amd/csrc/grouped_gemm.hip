// Products of rows with their expert's weights, and their gradients, in fp16 and
// bf16 on the matrix instructions:
//   out[r, n]       = sum_k a[r, k] W[e, n, k]         offsets[e] <= r < offsets[e + 1]
//   grad_a[r, k]    = sum_n grad[r, n] W[e, n, k]
//   grad_w[e, n, k] = sum_r grad[r, n] a[r, k]         over the rows r of expert e
// Products are exact, sums are fp32 in a fixed order, and a result is rounded
// once, at its store.  The operand that runs along the output's columns is the
// instruction's rows, so a lane ends with consecutive columns of one output row.
#include "grouped_tile.h"

namespace moe {
namespace {

// ------------------------------------------------------------- any alignment --
// Sizes, strides and addresses that the tile kernels' 16-byte loads do not take:
// a workgroup of four waves makes a tile of 64 x 64, 32 of the reduction at a
// time through registers into LDS, element by element at ragged ends.
constexpr int kAnyTile = 64, kAnyDepth = 32, kAnyRow = kAnyDepth + 8;

// An operand seen as [i, q], q along the reduction: one of its two strides is 1.
struct View {
  const uint16_t* base;
  int64_t ld;      // the other stride
  bool along;      // q is the contiguous one
  int n, depth;    // i < n, q < depth
};

__device__ __forceinline__ void any_load(const View& v, int i0, int q0,
                                         uint16_t (*tile)[kAnyRow]) {
  const int u = threadIdx.x;
  uint16_t e[8];
  const int i = i0 + (v.along ? u >> 2 : (u & 7) * 8), q = q0 + (v.along ? (u & 3) * 8 : u >> 3);
  const bool in = i < v.n && q < v.depth;
  const uint16_t* p = v.base + (v.along ? i * v.ld + q : q * v.ld + i);
  const int left = in ? (v.along ? v.depth - q : v.n - i) : 0;
  if (left >= 8) {
    const dwords4 d = load16(p);
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = static_cast<uint16_t>(d[j / 2] >> (16 * (j & 1)));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = j < left ? p[j] : uint16_t{0};
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (v.along)
      tile[u >> 2][(u & 3) * 8 + j] = e[j];
    else
      tile[(u & 7) * 8 + j][u >> 3] = e[j];
  }
}

template <Product P, typename T, typename TO>
__global__ __launch_bounds__(256) void grouped_any_kernel(GroupedArgs p, int col_tiles) {
  __shared__ __attribute__((aligned(16))) uint16_t xs[kAnyTile][kAnyRow], ys[kAnyTile][kAnyRow];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cols = P == Product::kOut ? p.N : p.K;
  int e, i0, i1, j0 = 0;
  View x, y;
  if constexpr (P == Product::kWeights) {
    const int row_tiles = (p.N + kAnyTile - 1) / kAnyTile;
    const int per = row_tiles * col_tiles;
    e = blockIdx.x / per;
    const int at = blockIdx.x - e * per;
    i0 = at / col_tiles * kAnyTile;
    i1 = min(p.N, i0 + kAnyTile);
    j0 = at % col_tiles * kAnyTile;
    int r0, r1;
    segment(p, e, r0, r1);
    const int n = max(r1 - r0, 0);
    x = View{p.x + r0 * p.x_ld, p.x_ld, false, p.N, n};
    y = View{p.y + r0 * p.y_ld, p.y_ld, false, p.K, n};
  } else {
    const int mt = blockIdx.x / col_tiles;
    j0 = (blockIdx.x - mt * col_tiles) * kAnyTile;
    if (!find_tile(count_tiles(p.offsets, p.E, p.rows, kAnyTile), mt, e, i0, i1)) return;
    const uint16_t* w = p.y + static_cast<int64_t>(e) * p.N * p.K;
    const int depth = P == Product::kOut ? p.K : p.N;
    x = View{p.x, p.x_ld, true, i1, depth};
    y = View{w, p.K, P == Product::kOut, cols, depth};
  }
  // wave w makes columns 16 w ... + 15 of all 64 rows
  const int col = lane & 15, g = lane >> 4;
  f32x4 acc[4] = {};
  for (int q = 0; q < x.depth; q += kAnyDepth) {
    any_load(x, i0, q, xs);
    any_load(y, j0, q, ys);
    __syncthreads();
    const dwords4 a = *reinterpret_cast<const dwords4*>(&ys[wave * 16 + col][8 * g]);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[i] = mfma16(T{}, a, *reinterpret_cast<const dwords4*>(&xs[i * 16 + col][8 * g]), acc[i]);
    __syncthreads();
  }
  const int j = j0 + wave * 16 + 4 * g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = i0 + i * 16 + col;
    if (row >= i1 || j >= cols) continue;
    if constexpr (P == Product::kWeights) {
      auto* o = static_cast<typename TO::bits*>(p.out) +
                (static_cast<int64_t>(e) * p.N + row) * p.K + j;
      f32x4 v = acc[i];
      if (p.accumulate) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (j + c < cols) v[c] += to_float(TO{}, o[c]);
      }
      store4<TO>(o, cols - j, v);
    } else {
      store4<TO>(static_cast<typename TO::bits*>(p.out) + row * p.out_ld + j, cols - j, acc[i]);
    }
  }
}

template <Product P>
void launch_any(const GroupedArgs& a, hipStream_t stream) {
  const int cols = P == Product::kOut ? a.N : a.K;
  const int col_tiles = (cols + kAnyTile - 1) / kAnyTile;
  const int64_t row_tiles =
      P == Product::kWeights ? static_cast<int64_t>(a.E) * ((a.N + kAnyTile - 1) / kAnyTile)
                             : a.rows / kAnyTile + (a.E < a.rows ? a.E : a.rows);
  const dim3 grid(static_cast<unsigned>(row_tiles * col_tiles));
  with_types(a, [&](auto t, auto to) {
    hipLaunchKernelGGL((grouped_any_kernel<P, decltype(t), decltype(to)>), grid, dim3(256), 0,
                       stream, a, col_tiles);
  });
}

}  // namespace

// What the tile kernels' 16-byte loads and 32-bit offsets take.
static bool tiles_take(Product p, const GroupedArgs& a) {
  auto whole = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 15u) == 0; };
  constexpr int64_t kMaxLd = 1 << 20;
  if (a.N % 8 || a.K % 8 || a.x_ld % 8 || a.x_ld > kMaxLd || !whole(a.x) || !whole(a.y)) return false;
  return p != Product::kWeights || (a.y_ld % 8 == 0 && a.y_ld <= kMaxLd);
}

void launch_grouped(Product p, const GroupedArgs& a, hipStream_t stream) {
  const bool tiles = tiles_take(p, a);
  switch (p) {
    case Product::kOut: return tiles ? launch_grouped_out(a, stream) : launch_any<Product::kOut>(a, stream);
    case Product::kRows: return tiles ? launch_grouped_rows(a, stream) : launch_any<Product::kRows>(a, stream);
    case Product::kWeights:
      return tiles ? launch_grouped_weights(a, stream) : launch_any<Product::kWeights>(a, stream);
  }
}

}  // namespace moe
