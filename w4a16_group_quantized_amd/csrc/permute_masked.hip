// Stable sort of the S = T * top_k slots by expert that leaves slots out: an
// id outside [first, first + E) drops its slot (padding tokens, experts held
// by other ranks).  A token may name an expert more than once.
//
// A counting sort in chunks of 1024 slots, one workgroup of 16 waves each, one
// slot per lane.  Inside a wave, equal experts are found by one ballot per bit
// of the expert number; the waves then add to the chunk's LDS counts in wave
// order (a barrier between them), so the rank of a slot in its chunk counts
// the earlier slots only and nothing depends on which wave runs first.
//   one chunk           one launch does everything
//   up to kFewChunks    ranks and counts, then a scatter in which every
//                       workgroup sums the counts of all chunks itself (they
//                       are in L2: 40 chunks x 512 experts are 80 KB), which
//                       takes the scan's launch out
//   more                a scan launch between them, its work linear in the
//                       chunks
// Bound by latency: 4.7 us for 80 slots, 9.8 us a call for 40960 slots of 512 experts
// (40 chunks: two launches, 4.0 and 5.5 us at best and 4.5 and 6.0 on average in the
// kernel trace).
#include "mxfp4.h"
#include "permute.h"

namespace moe {
namespace {

constexpr int kChunk = kScanThreads;
constexpr int kFewChunks = 64;

// Rank of this thread's slot among the chunk's earlier slots of the same
// expert (expert < 0: none); leaves the chunk's counts in hist[0, E).
__device__ __forceinline__ int chunk_ranks(int expert, int E, int* hist) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < E; e += kChunk) hist[e] = 0;
  unsigned long long peers = __ballot(expert >= 0);
  for (int b = 0; (E - 1) >> b; ++b) {
    const unsigned long long on = __ballot((expert >> b) & 1);
    peers &= ((expert >> b) & 1) ? on : ~on;
  }
  const int before = __popcll(peers & ((1ull << lane) - 1ull));
  int rank = -1;
  for (int w = 0; w < kChunk / 64; ++w) {
    __syncthreads();
    if (wave == w && expert >= 0) {
      const int base = hist[expert];
      rank = base + before;
      if (before + 1 == __popcll(peers)) hist[expert] = rank + 1;  // the last peer
    }
  }
  __syncthreads();
  return rank;
}

__device__ __forceinline__ int slot_expert(const int* ids, int s, int S, int first, int E) {
  if (s >= S) return -1;
  const uint32_t e = static_cast<uint32_t>(ids[s]) - static_cast<uint32_t>(first);
  return e < static_cast<uint32_t>(E) ? static_cast<int>(e) : -1;
}

// Offsets of all experts (returned for this thread's experts per * tid + i)
// and the number of rows kept; workgroup 0 writes offsets and active list.
__device__ __forceinline__ int scan_experts(const int (&cnt)[kPerThread], int per, int E,
                                            bool write, int* offsets, int* active, int* num_active,
                                            int* wave_tot, int (&off)[kPerThread]) {
  const int tid = threadIdx.x;
  int csum = 0, fsum = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    csum += cnt[i];
    fsum += cnt[i] > 0;
  }
  int kept, found;
  int cpre = block_exclusive_scan(csum, wave_tot, kept);
  int fpre = block_exclusive_scan(fsum, wave_tot, found);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int e = per * tid + i;
    off[i] = cpre;
    if (write && i < per && e < E) {
      offsets[e] = cpre;
      if (cnt[i] > 0) active[fpre++] = e;
    }
    cpre += cnt[i];
  }
  if (write) {
    for (int e = found + tid; e < E; e += kScanThreads) active[e] = -1;
    if (tid == 0) {
      offsets[E] = kept;
      *num_active = found;
    }
  }
  return kept;
}

__global__ __launch_bounds__(kChunk) void masked_single_kernel(
    const int* __restrict__ ids, int S, int first, int E, int* __restrict__ offsets,
    int* __restrict__ sorted_slots, int* __restrict__ slot_rows, int* __restrict__ active,
    int* __restrict__ num_active) {
  __shared__ int hist[kMaxExperts];
  __shared__ int wave_tot[kChunk / 64 + 1];
  const int s = threadIdx.x;
  const int expert = slot_expert(ids, s, S, first, E);
  const int rank = chunk_ranks(expert, E, hist);
  const int per = (E + kChunk - 1) / kChunk;
  int cnt[kPerThread], off[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int e = per * s + i;
    cnt[i] = i < per && e < E ? hist[e] : 0;
  }
  const int kept = scan_experts(cnt, per, E, true, offsets, active, num_active, wave_tot, off);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int e = per * s + i;
    if (i < per && e < E) hist[e] = off[i];
  }
  __syncthreads();
  if (s >= S) return;
  const int row = expert >= 0 ? hist[expert] + rank : -1;
  slot_rows[s] = row;
  if (row >= 0) sorted_slots[row] = s;
  if (s >= kept) sorted_slots[s] = -1;
}

// Ranks into slot_rows, counts of the chunk into counts[chunk, E).
__global__ __launch_bounds__(kChunk) void masked_rank_kernel(const int* __restrict__ ids, int S,
                                                             int first, int E,
                                                             int* __restrict__ slot_rows,
                                                             int* __restrict__ counts) {
  __shared__ int hist[kMaxExperts];
  const int s = blockIdx.x * kChunk + threadIdx.x;
  const int expert = slot_expert(ids, s, S, first, E);
  const int rank = chunk_ranks(expert, E, hist);
  if (s < S) slot_rows[s] = rank;
  for (int e = threadIdx.x; e < E; e += kChunk)
    counts[static_cast<size_t>(blockIdx.x) * E + e] = hist[e];
}

// Counts to rows in earlier chunks, in place, one thread per expert; the
// totals of the experts into totals[0, E).
__global__ __launch_bounds__(256) void masked_scan_kernel(int chunks, int E,
                                                          int* __restrict__ counts,
                                                          int* __restrict__ totals) {
  const int e = blockIdx.x * 256 + threadIdx.x;
  if (e >= E) return;
  int run = 0;
  for (int c0 = 0; c0 < chunks; c0 += 16) {
    int c[16];
#pragma unroll
    for (int u = 0; u < 16; ++u)
      c[u] = c0 + u < chunks ? counts[static_cast<size_t>(c0 + u) * E + e] : 0;
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      if (c0 + u < chunks) counts[static_cast<size_t>(c0 + u) * E + e] = run;
      run += c[u];
    }
  }
  totals[e] = run;
}

// SCANNED: counts hold rows in earlier chunks and totals the experts' rows;
// otherwise both are summed here.
template <bool SCANNED>
__global__ __launch_bounds__(kChunk) void masked_scatter_kernel(
    const int* __restrict__ ids, int S, int first, int E, int chunks,
    const int* __restrict__ counts, const int* __restrict__ totals, int* __restrict__ offsets,
    int* __restrict__ sorted_slots, int* __restrict__ slot_rows, int* __restrict__ active,
    int* __restrict__ num_active) {
  __shared__ int seg[kMaxExperts];
  __shared__ int wave_tot[kChunk / 64 + 1];
  const int chunk = blockIdx.x;
  const int per = (E + kChunk - 1) / kChunk;
  int cnt[kPerThread], before[kPerThread], off[kPerThread];
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int e = per * threadIdx.x + i;
    cnt[i] = before[i] = 0;
    if (i < per && e < E) {
      if constexpr (SCANNED) {
        cnt[i] = totals[e];
        before[i] = counts[static_cast<size_t>(chunk) * E + e];
      } else {
#pragma unroll 8
        for (int c = 0; c < chunks; ++c) {
          const int n = counts[static_cast<size_t>(c) * E + e];
          cnt[i] += n;
          before[i] += c < chunk ? n : 0;
        }
      }
    }
  }
  const int kept =
      scan_experts(cnt, per, E, chunk == 0, offsets, active, num_active, wave_tot, off);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int e = per * threadIdx.x + i;
    if (i < per && e < E) seg[e] = off[i] + before[i];
  }
  __syncthreads();
  const int s = chunk * kChunk + threadIdx.x;
  if (s >= S) return;
  const int expert = slot_expert(ids, s, S, first, E);
  if (expert >= 0) {
    const int row = seg[expert] + slot_rows[s];
    slot_rows[s] = row;
    sorted_slots[row] = s;
  }
  if (s >= kept) sorted_slots[s] = -1;
}

int64_t chunks_of(int64_t S) { return (S + kChunk - 1) / kChunk; }

}  // namespace

size_t permute_masked_workspace_bytes(int64_t T, int top_k, int E) {
  const int64_t chunks = chunks_of(T * top_k);
  return chunks <= 1 ? 0 : static_cast<size_t>(chunks + 1) * E * sizeof(int);
}

void launch_permute_masked(const int* ids, int T, int top_k, int first, int E, int* offsets,
                           int* sorted_slots, int* slot_rows, int* active, int* num_active,
                           void* workspace, hipStream_t stream) {
  const int S = T * top_k;
  const int chunks = static_cast<int>(chunks_of(S));
  if (chunks == 1) {
    hipLaunchKernelGGL(masked_single_kernel, dim3(1), dim3(kChunk), 0, stream, ids, S, first, E,
                       offsets, sorted_slots, slot_rows, active, num_active);
    return;
  }
  int* counts = static_cast<int*>(workspace);
  int* totals = counts + static_cast<size_t>(chunks) * E;
  hipLaunchKernelGGL(masked_rank_kernel, dim3(chunks), dim3(kChunk), 0, stream, ids, S, first, E,
                     slot_rows, counts);
  if (chunks <= kFewChunks) {
    hipLaunchKernelGGL(masked_scatter_kernel<false>, dim3(chunks), dim3(kChunk), 0, stream, ids, S,
                       first, E, chunks, counts, totals, offsets, sorted_slots, slot_rows, active,
                       num_active);
    return;
  }
  hipLaunchKernelGGL(masked_scan_kernel, dim3((E + 255) / 256), dim3(256), 0, stream, chunks, E,
                     counts, totals);
  hipLaunchKernelGGL(masked_scatter_kernel<true>, dim3(chunks), dim3(kChunk), 0, stream, ids, S,
                     first, E, chunks, counts, totals, offsets, sorted_slots, slot_rows, active,
                     num_active);
}

}  // namespace moe
