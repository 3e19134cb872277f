// Slots of tokens sorted by expert (the definition is at moe_decode_sort_slots in
// include/moe_decode.h): a counting sort that keeps the slots' order.
//
// The slots are cut into parts of whole rounds of 64 for each of 16 wavefronts.  A
// slot's rank among those of its expert in its round comes from ballots, one for each bit
// of the expert's number; its place is that, plus the expert's slots in earlier
// rounds, wavefronts and parts, plus the slots of earlier experts.
// Up to 8192 slots one launch does it: each part counts the slots of all others for
// itself, which costs less than a launch.  Beyond, a first launch counts each part's slots
// of each expert, and the parts of the second add up what lies before them.  Counts
// are added in LDS by one lane for all of its round that share its expert: lanes of one
// address are served one after another (32768 slots counted lane by lane 20 us).
// Latencies bound it: 32768 slots of 128 experts 3.6 + 5.2 us, 8192 of 9 in one launch 7.2.
#pragma once

#include "prims.hpp"

namespace moe {

constexpr int kSortThreads = 1024;
constexpr int kSortWaves = kSortThreads / 64;
constexpr int kSortExperts = 1024;      // E limit
constexpr int kSortOnce = 8192;         // slots up to which one launch does it (their numbers fit in 16 bits)
constexpr int kSortMostParts = 256;

__host__ __device__ constexpr int sort_parts(int slots) {
  const int n = (slots - 1) / kSortThreads + 1;
  return n < kSortMostParts ? n : kSortMostParts;
}
// Integers of workspace for the parts' counts.
__host__ __device__ constexpr size_t sort_counts(int slots, int E) {
  return slots <= kSortOnce ? 0 : (size_t)sort_parts(slots) * E;
}
// Slots of one part: whole rounds of all wavefronts.
__host__ __device__ constexpr int sort_part(int slots) {
  const int rounds = (slots - 1) / (sort_parts(slots) * kSortThreads) + 1;
  return rounds * kSortThreads;
}

struct SortArgs {
  const int32_t* ids;
  const uint8_t* valid;
  int32_t* counts;
  int32_t* x_rows;
  int32_t* positions;
  int32_t* before;   // [parts, E] slots of each expert in each part, where there are more than kSortOnce
  int slots, E, k, part;
  uint32_t magic;    // ceil(2^32 / k)
  bool rest;         // ids outside [0, E - 1) are of the last expert
};

__device__ __forceinline__ int sort_token(const SortArgs& a, int s) {
  if (a.k == 1) return s;
  const int q = (int)__umulhi((uint32_t)s, a.magic);   // the quotient, or one more
  return q - (q * a.k > s ? 1 : 0);
}
// The expert of slot s; -1 where it is not counted.  The loads are always made, of a slot that is there: one under a
// condition of the lane's would be waited for at its end.
__device__ __forceinline__ int sort_expert(const SortArgs& a, int s, int end) {
  const int from = min(s, a.slots - 1), e = a.ids[from];
  if (a.rest) return s >= end ? -1 : (unsigned)e < (unsigned)(a.E - 1) ? e : a.E - 1;
  const bool on = !a.valid || a.valid[sort_token(a, from)] != 0;
  return (on & (s < end) & ((unsigned)e < (unsigned)a.E)) ? e : -1;
}

// A round of 64 slots: the lanes that share this lane's expert (< 1 << bits).
__device__ __forceinline__ uint64_t sort_peers(int e, int bits) {
  uint64_t same = __builtin_amdgcn_ballot_w64(e >= 0);
  // all of one: rows of a prompt
  if (__builtin_amdgcn_ballot_w64(e == __builtin_amdgcn_readfirstlane(e)) == ~0ull) return same;
  for (int b = 0; b < bits; ++b) {
    const uint64_t ones = __builtin_amdgcn_ballot_w64(e >> b & 1);
    same &= e >> b & 1 ? ones : ~ones;
  }
  return same;
}
__device__ __forceinline__ int sort_bits(int E) { return E > 1 ? 32 - __builtin_clz(E - 1) : 0; }
// One lane of them, the last.
__device__ __forceinline__ bool sort_speaks(uint64_t same, int lane) { return same >> lane == 1; }

static __global__ __launch_bounds__(kSortThreads) void sort_count_kernel(SortArgs a) {
  __shared__ int32_t hist[kSortExperts];
  const int tid = threadIdx.x, lane = tid & 63, bits = sort_bits(a.E);
  const int s0 = (int)blockIdx.x * a.part, s1 = min(a.slots - s0, a.part) + s0;
  if (tid < a.E) hist[tid] = 0;
  int e = sort_expert(a, s0 + tid, s1);
  __syncthreads();
  for (int s = s0 + tid; s - lane < s1; s += kSortThreads) {   // whole wavefronts
    const int next = sort_expert(a, s + kSortThreads, s1);
    const uint64_t same = sort_peers(e, bits);
    if (e >= 0 && sort_speaks(same, lane)) atomicAdd(&hist[e], __builtin_popcountll(same));
    e = next;
  }
  __syncthreads();
  if (tid < a.E) a.before[(size_t)blockIdx.x * a.E + tid] = hist[tid];
}

// ONCE: the parts count for themselves.  SINGLE: a wavefront has one round.
template <bool ONCE, bool SINGLE>
static __global__ __launch_bounds__(kSortThreads) void sort_place_kernel(SortArgs a) {
  __shared__ uint16_t wave_count[kSortWaves][kSortExperts];   // of the part: fewer than 2^16 in each wavefront's share
  __shared__ uint32_t seen[kSortExperts];   // slots of an expert, and of them before this part: in ONCE's one word, or
  __shared__ uint32_t seen_before[ONCE ? 1 : kSortExperts];   // in two
  __shared__ int32_t start[kSortExperts];   // where the part's slots of each expert begin
  __shared__ int32_t sums[kSortWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int s0 = (int)blockIdx.x * a.part, s1 = min(a.slots - s0, a.part) + s0;
  const int share = a.part / kSortWaves, w0 = s0 + w * share;   // this wavefront's slots
  const int w1 = min(w0 + share, s1);
  constexpr int U = ONCE ? kSortOnce / kSortThreads : 1;   // the parts; ONCE: a slot of each, requested together
  int parts_e[U], mine_e = -1;
  if constexpr (ONCE) {
#pragma unroll
    for (int u = 0; u < U; ++u) parts_e[u] = sort_expert(a, u * kSortThreads + tid, a.slots);
  } else if constexpr (SINGLE) {
    mine_e = sort_expert(a, w0 + lane, w1);
  }
  if (tid < a.E) {
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) wave_count[i][tid] = 0;
    seen[tid] = 0;
    if (!ONCE) seen_before[tid] = 0;
  }
  const int bits = sort_bits(a.E);
  __syncthreads();

  uint64_t mine_same = 0;
  if constexpr (ONCE) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u * kSortThreads >= a.slots) break;
      const int e = parts_e[u];
      const uint64_t same = sort_peers(e, bits);
      const uint32_t n = (uint32_t)__builtin_popcountll(same);
      if (e >= 0 && sort_speaks(same, lane)) {
        atomicAdd(&seen[e], n << 16 | (u < (int)blockIdx.x ? n : 0u));
        if (u == (int)blockIdx.x) wave_count[w][e] = (uint16_t)n;
      }
      if (u == (int)blockIdx.x) {
        mine_e = e;
        mine_same = same;
      }
    }
  } else {
    for (int s = w0; s < w1; s += 64) {
      const int e = SINGLE ? mine_e : sort_expert(a, s + lane, w1);
      const uint64_t same = sort_peers(e, bits);
      if (SINGLE) mine_same = same;
      if (e >= 0 && sort_speaks(same, lane)) wave_count[w][e] += (uint16_t)__builtin_popcountll(same);
    }
    // 1024 threads share out the parts' counts: several threads an expert where there are fewer experts
    const int stride = 1 << bits, first = tid >> bits, e = tid & (stride - 1);
    uint32_t n = 0, before = 0;
    if (e < a.E) {
#pragma unroll 8
      for (int i = first; i < (int)gridDim.x; i += kSortThreads >> bits) {
        const uint32_t c = (uint32_t)a.before[(size_t)i * a.E + e];
        n += c;
        before += i < (int)blockIdx.x ? c : 0u;
      }
      atomicAdd(&seen[e], n);
      atomicAdd(&seen_before[e], before);
    }
  }
  __syncthreads();
  // thread e holds expert e
  int total = 0, mine = 0;
  if (tid < a.E) {
    total = (int)(ONCE ? seen[tid] >> 16 : seen[tid]);
    mine = (int)(ONCE ? seen[tid] & 0xFFFFu : seen_before[tid]);
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
    const int e = SINGLE ? mine_e : sort_expert(a, s + lane, w1);
    const uint64_t same = SINGLE ? mine_same : sort_peers(e, bits);
    if (s + lane < w1) {
      int at = -1;
      if (e >= 0) {
        at = start[e] + wave_count[w][e] + __builtin_popcountll(same & ((1ull << lane) - 1));
        a.x_rows[at] = sort_token(a, s + lane);
      }
      if (a.positions) a.positions[s + lane] = at;
    }
    if (!SINGLE) {
      __builtin_amdgcn_wave_barrier();   // all have read before the last of them adds
      if (e >= 0 && sort_speaks(same, lane)) wave_count[w][e] += (uint16_t)__builtin_popcountll(same);
      __builtin_amdgcn_wave_barrier();
    }
  }
  for (int s = max(s0, all) + tid; s < s1; s += kSortThreads) a.x_rows[s] = -1;   // behind the last expert's
}

// The one launch, or both.
inline void launch_sort(hipStream_t st, const SortArgs& a) {
  const dim3 grid((unsigned)sort_parts(a.slots)), block(kSortThreads);
  if (a.slots <= kSortOnce) {
    hipLaunchKernelGGL((sort_place_kernel<true, true>), grid, block, 0, st, a);
    return;
  }
  hipLaunchKernelGGL(sort_count_kernel, grid, block, 0, st, a);
  if (a.part == kSortThreads) hipLaunchKernelGGL((sort_place_kernel<false, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((sort_place_kernel<false, false>), grid, block, 0, st, a);
}

}  // namespace moe
