// The gradient of the weights on the tile kernel (grouped_tile.h).
#include "grouped_tile.h"

namespace moe {
namespace {

int64_t tiles_of(int64_t blocks, int N, int K, int size) {
  return blocks * ((N + size - 1) / size) * ((K + size - 1) / size);
}

// Tiles of 256 where they do not hang over the matrix by more than an eighth: 128 experts
// of 1280 x 640, 8000 rows, 50 us, with tiles of 128 x 128 46; 512 of 1280 x 2560, 40960
// rows, 840 and 1076; 8 of 8192 x 4096, 16381 rows, 861 and 1073.
int size_of(int64_t blocks, int N, int K) {
  const bool fits = tiles_of(1, N, K, 256) * 65536 <= static_cast<int64_t>(N) * K / 8 * 9;
  const auto tiles = [&](int size) { return tiles_of(blocks, N, K, size); };
  const int size = pick_size(tiles);
  if (size != 256 || (fits && tiles(256) >= kUnits)) return size;
  return cost_of(128, tiles(128)) <= cost_of(64, tiles(64)) ? 128 : 64;
}

// Few tiles of a long sum: its rows are shared out to parts, whose sums a second kernel
// adds.  Parts have 256 rows at least, and are taken where the shorter sums save more than
// the second launch and the way of the parts through memory cost: 1 expert of 512 x 2560,
// 4096 rows: 25 us, in one part 30; 40960 rows: 139 and 312; 64 x 64, 40960 rows: 14.5
// and 187; 8 experts of 256 x 512, 20000 rows: four parts 20.2, one 15.5.
int parts_of(int64_t rows, int E, int N, int K) {
  constexpr int64_t kLaunch = 600, kBytesPerUnit = 50000;  // 6 us; 5 TB/s
  const auto cost = [&](int64_t parts) {
    const int64_t blocks = E * parts;
    const int size = size_of(blocks, N, K);
    const int64_t chunks = (rows / blocks + kChunk - 1) / kChunk;
    const int64_t sums = chunks * cost_of(size, tiles_of(blocks, N, K, size));
    return parts == 1 ? sums : sums + kLaunch + blocks * N * K * 4 / kBytesPerUnit;
  };
  int64_t best = 1, least = cost(1);
  for (int64_t parts = 2; parts <= 32 && parts * E * 256 <= rows; ++parts) {
    const int64_t c = cost(parts);
    if (c < least) best = parts, least = c;
  }
  return static_cast<int>(best);
}

// out = (what it holds +) the parts' sums, parts ascending; 4 elements per thread, of the
// expert blockIdx.y.  Nothing here needs more than an element's alignment.
template <typename TO>
__global__ __launch_bounds__(256) void add_parts_kernel(const float* __restrict__ sums, int parts,
                                                        int64_t n, int accumulate,
                                                        typename TO::bits* __restrict__ out) {
  const int64_t at = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (at >= n) return;
  const int left = static_cast<int>(min(n - at, int64_t{4}));
  const float* from = sums + blockIdx.y * parts * n + at;
  out += blockIdx.y * n + at;
  f32x4 v{};
  if (accumulate) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) v[i] = to_float(TO{}, out[i]);
  }
  if (left == 4) {
#pragma unroll 8
    for (int p = 0; p < parts; ++p) v += __builtin_bit_cast(f32x4, load16(from + p * n));
  } else {
    for (int p = 0; p < parts; ++p)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) v[i] += from[p * n + i];
  }
  store4<TO>(out, left, v);
}

}  // namespace

size_t grouped_workspace_bytes(int64_t rows, int E, int N, int K) {
  const int parts = parts_of(rows, E, N, K);
  return parts > 1 ? static_cast<size_t>(E) * parts * N * K * sizeof(float) : 0;
}

GroupedArgs grouped_part_sums(const GroupedArgs& a) {
  GroupedArgs b = a;
  b.parts = parts_of(a.rows, a.E, a.N, a.K);
  b.by_parts = Divisor(b.parts);
  if (b.parts > 1) {
    b.out = a.partial;
    b.out_dtype = MOE_F32;
    b.accumulate = 0;
  }
  return b;
}

void launch_add_parts(const GroupedArgs& a, int parts, hipStream_t stream) {
  if (parts == 1) return;
  const int64_t n = static_cast<int64_t>(a.N) * a.K;
  const dim3 grid(static_cast<unsigned>((n + 1023) / 1024), a.E);
  with_dtype(a.out_dtype, [&](auto to) {
    using TO = decltype(to);
    hipLaunchKernelGGL((add_parts_kernel<TO>), grid, dim3(256), 0, stream, a.partial, parts, n,
                       a.accumulate, static_cast<typename TO::bits*>(a.out));
  });
}

void launch_grouped_weights(const GroupedArgs& a, hipStream_t stream) {
  const GroupedArgs b = grouped_part_sums(a);
  const int size = size_of(static_cast<int64_t>(a.E) * b.parts, a.N, a.K);
  if (size == 256)
    launch_grouped_tiles<Grouped256, Product::kWeights>(b, stream);
  else if (size == 128)
    launch_grouped_tiles<Grouped128, Product::kWeights>(b, stream);
  else
    launch_grouped_tiles<Grouped64, Product::kWeights>(b, stream);
  launch_add_parts(a, b.parts, stream);
}

}  // namespace moe
