// Slots of tokens sorted by expert (the definition is at moe_decode_sort_slots in
// include/moe_decode.h): a counting sort that keeps the slots' order.
//
// The slots are cut into parts of whole rounds of 64 for each wavefront.  A slot's
// rank among those of its expert in its round comes from ballots, one for each bit
// of the expert's number; its place is that, plus the expert's slots in earlier
// rounds, wavefronts and parts, plus the slots of earlier experts.
// One part: one launch.  More: a first launch counts each part's slots of each
// expert, and every part of the second adds up what lies before it.
#pragma once

#include "prims.hpp"

namespace moe {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortExperts = 1024;      // E limit
constexpr int kSortAlone = 4096;        // slots that one workgroup takes without a second launch
constexpr int kSortMostParts = 256;

__host__ __device__ constexpr int sort_parts(int slots) {
  if (slots <= kSortAlone) return 1;
  const int n = (slots + 2 * kSortThreads - 1) / (2 * kSortThreads);
  return n < kSortMostParts ? n : kSortMostParts;
}
// Slots of one part: whole rounds of all wavefronts.
__host__ __device__ constexpr int sort_part(int slots) {
  const int parts = sort_parts(slots);
  const int rounds = (slots - 1) / (parts * kSortThreads) + 1;
  return rounds * kSortThreads;
}

struct SortArgs {
  const int32_t* ids;
  const uint8_t* valid;
  int32_t* counts;
  int32_t* x_rows;
  int32_t* positions;
  int32_t* before;   // [parts, E] slots of each expert in each part
  int slots, E, k, part;
  uint32_t magic;    // ceil(2^32 / k)
  bool rest;         // ids outside [0, E - 1) are of the last expert
};

__device__ __forceinline__ int sort_token(const SortArgs& a, int s) {
  if (a.k == 1) return s;
  const int q = (int)__umulhi((uint32_t)s, a.magic);   // the quotient, or one more
  return q - (q * a.k > s ? 1 : 0);
}
// The expert of slot s; -1 where it is not counted.
__device__ __forceinline__ int sort_expert(const SortArgs& a, int s, int end) {
  if (s >= end) return -1;
  const int e = a.ids[s];
  if (a.rest) return (unsigned)e < (unsigned)(a.E - 1) ? e : a.E - 1;
  const bool on = (unsigned)e < (unsigned)a.E && (!a.valid || a.valid[sort_token(a, s)]);
  return on ? e : -1;
}

static __global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ int32_t hist[kSortExperts];
  const int tid = threadIdx.x;
  const int s0 = (int)blockIdx.x * a.part, s1 = min(a.slots - s0, a.part) + s0;
  for (int e = tid; e < a.E; e += kSortThreads) hist[e] = 0;
  __syncthreads();
  for (int s = s0 + tid; s < s1; s += kSortThreads) {
    const int e = sort_expert(a, s, s1);
    if (e >= 0) atomicAdd(&hist[e], 1);
  }
  __syncthreads();
  for (int e = tid; e < a.E; e += kSortThreads) a.before[(size_t)blockIdx.x * a.E + e] = hist[e];
}

// ALONE: there is no other part.
template <bool ALONE>
static __global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  __shared__ uint16_t wave_count[kSortWaves][kSortExperts];   // of the part: fewer than 2^16 in each wavefront's share
  __shared__ int32_t start[kSortExperts];   // where the part's slots of each expert begin
  __shared__ int32_t sums[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int s0 = (int)blockIdx.x * a.part, s1 = min(a.slots - s0, a.part) + s0;
  const int share = a.part / kSortWaves, w0 = s0 + w * share;   // this wavefront's slots
  const int w1 = min(w0 + share, s1);
  for (int i = tid; i < kSortWaves * a.E; i += kSortThreads) wave_count[i / a.E][i % a.E] = 0;
  int bits = 0;
  while ((1 << bits) < a.E) ++bits;
  __syncthreads();

  // a round of 64 slots: the lanes that share this lane's expert
  auto peers = [&](int e) {
    uint64_t same = __builtin_amdgcn_ballot_w64(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const uint64_t ones = __builtin_amdgcn_ballot_w64(e >> b & 1);
      same &= e >> b & 1 ? ones : ~ones;
    }
    return same;
  };
  for (int s = w0; s < w1; s += 64) {
    const int e = sort_expert(a, s + lane, w1);
    const uint64_t same = peers(e);
    if (e >= 0 && (same >> lane) == 1) wave_count[w][e] += (uint16_t)__builtin_popcountll(same);   // the last of them
  }
  __syncthreads();
  // experts' totals and what lies before this part; thread e holds expert e
  int total = 0, mine = 0;
  if (tid < a.E) {
    if constexpr (ALONE) {
#pragma unroll
      for (int i = 0; i < kSortWaves; ++i) total += wave_count[i][tid];
    } else {
      const int parts = (int)gridDim.x;
      for (int i = 0; i < parts; ++i) {
        const int n = a.before[(size_t)i * a.E + tid];
        mine += i < (int)blockIdx.x ? n : 0;
        total += n;
      }
    }
  }
  const int upto = wave_incl_scan(total);
  if (lane == 63) sums[w] = upto;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kSortWaves; ++i) {
    base += i < w ? sums[i] : 0;
    all += sums[i];
  }
  if (tid < a.E) {
    start[tid] = base + upto - total + mine;
    if (blockIdx.x == 0) a.counts[tid] = total;
    int run = 0;
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) {   // counts -> what the part's earlier wavefronts have
      const int n = wave_count[i][tid];
      wave_count[i][tid] = (uint16_t)run;
      run += n;
    }
  }
  __syncthreads();
  for (int s = w0; s < w1; s += 64) {
    const int e = sort_expert(a, s + lane, w1);
    const uint64_t same = peers(e);
    if (s + lane < w1) {
      int at = -1;
      if (e >= 0) {
        at = start[e] + wave_count[w][e] + __builtin_popcountll(same & ((1ull << lane) - 1));
        a.x_rows[at] = sort_token(a, s + lane);
      }
      if (a.positions) a.positions[s + lane] = at;
    }
    __builtin_amdgcn_wave_barrier();   // all have read before the last of them adds
    if (e >= 0 && (same >> lane) == 1) wave_count[w][e] += (uint16_t)__builtin_popcountll(same);
    __builtin_amdgcn_wave_barrier();
  }
  for (int s = max(s0, all) + tid; s < s1; s += kSortThreads) a.x_rows[s] = -1;   // behind the last expert's
}

// Both launches (or the one), of `parts` workgroups.
inline void launch_sort(hipStream_t st, const SortArgs& a, int parts) {
  const dim3 grid((unsigned)parts), block(kSortThreads);
  if (parts == 1) {
    hipLaunchKernelGGL(sort_place_kernel<true>, grid, block, 0, st, a);
  } else {
    hipLaunchKernelGGL(sort_count_kernel, grid, block, 0, st, a);
    hipLaunchKernelGGL(sort_place_kernel<false>, grid, block, 0, st, a);
  }
}

}  // namespace moe
