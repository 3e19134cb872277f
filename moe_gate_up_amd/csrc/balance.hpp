// Router training: per-expert counts, the balance and z losses, and their
// gradient with respect to the logits (the formulas are at
// moe_decode_balance in include/moe_decode.h).
//
// Both passes stream the logits once.  A row's softmax lives in registers:
// LR lanes (16 up to 256 experts, else 64) hold V logits each, so one
// wavefront works on 64 / LR rows at a time and the row's maximum and sums are
// V - 1 operations in the lane and 4 (or 6) DPP steps across it.  With 16
// lanes a row of 128 experts is two 16-byte loads per lane.
//
// The next round of rows is requested before the current one is worked on.
//
// Forward: a workgroup takes a part of one group's tokens; each
// lane adds up its columns' probabilities over its rows, the wavefronts' sums
// are added in LDS in a fixed order, and the slots are counted with integer
// LDS atomics, whose order cannot change the result.  The parts' sums go to
// the workspace, and a second launch adds them (FP64, fixed order); a single
// part (up to 256 tokens) finishes alone.
// Backward: the same walk with f_ge in registers; the softmax is computed
// again rather than stored (a stored one would be T E more bytes each way).
//
// 262144 tokens of 128 experts, FP32, 64 padded groups: both passes 74 us for
// 410 MB (5.5 TB/s; a copy of that size 6.3), the forward pass alone 33, of them 7
// the second launch: memory, and about 120 vector instructions for 4 rows.  With
// its counting left out the forward pass is 1.5 us faster.  More wavefronts (1024
// parts: 12 us slower) or a second round requested ahead (the same) do not help.
// 4096 tokens: 4.1, 4.2 and 4.2 us for the three launches, which is their latency.
#pragma once

#include "prims.hpp"
#include "router.hpp"

namespace moe {

constexpr int kBalThreads = 512;
constexpr int kBalWaves = kBalThreads / 64;
constexpr int kBalMaxExperts = 1024;
constexpr int kBalMaxK = 64;
constexpr int kBalSumThreads = 1024;
constexpr int kBalSumWaves = kBalSumThreads / 64;
constexpr int kBalSumCols = 32;       // experts that one workgroup of the second launch adds up, at least
constexpr int kBalTargetParts = 512;  // workgroups of a pass: 2 per CU
constexpr int kBalAlone = 256;        // tokens that one workgroup takes without a second launch

constexpr int kBalMostTokens = 32768; // tokens of a part: what is added up in FP32
constexpr int kBalMaxTokens = 1 << 30; // T: token numbers a round past the last one are 32-bit too

// Parts each group's tokens are cut into: enough workgroups for the chip, of
// at least 32 tokens each and few enough for FP32 sums.
__host__ __device__ constexpr int balance_parts(int S, int G) {
  if ((long long)S * G <= kBalAlone) return 1;
  const int by_chip = (kBalTargetParts + G - 1) / G;
  const int by_sums = (S + kBalMostTokens - 1) / kBalMostTokens;
  const int by_work = (S + 31) / 32;
  const int parts = by_chip > by_sums ? by_chip : by_sums;
  return parts < by_work ? parts : by_work;
}

__host__ __device__ constexpr int balance_splits(int E) { return (E + kBalSumCols - 1) / kBalSumCols; }

// Workspace: the parts' probability sums and counts [G parts, E], z sums and
// valid tokens [G parts]; the second launch's sums [G, splits] and its ticket.
struct BalanceLayout {
  size_t psum, cnt, z, n, dot, zsum, ticket, total;
  __host__ __device__ BalanceLayout(long long S, int E, int G) {
    const size_t rows = (size_t)G * balance_parts((int)S, G);
    size_t o = 0;
    auto take = [&](size_t b) { const size_t r = o; o += (b + 255) & ~(size_t)255; return r; };
    psum = take(rows * E * 4);
    cnt = take(rows * E * 4);
    z = take(rows * 4);
    n = take(rows * 4);
    dot = take((size_t)G * balance_splits(E) * 8);
    zsum = take((size_t)G * 8);
    ticket = take(4);
    total = o;
  }
};

template <int LR>
__device__ __forceinline__ float row_sum(float v) {
  if constexpr (LR == 16) return row_sum16(v);
  return wave_sum_f32(v);
}

// Maximum over the row's lanes (v_max_f32: a NaN loses against a number).
template <int LR>
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, dpp<0xB1>(v));
  v = fmaxf(v, dpp<0x4E>(v));
  v = fmaxf(v, dpp<0x141>(v));
  v = fmaxf(v, dpp<0x140>(v));
  if constexpr (LR == 64) {
    v = fmaxf(v, __shfl_xor(v, 16));
    v = fmaxf(v, __shfl_xor(v, 32));
  }
  return v;
}

// The columns of lane `l` of a row: groups of C consecutive ones (C = 4 with
// whole 4-element loads, else 1), LR groups apart.
template <int LR, int C>
__device__ __forceinline__ int balance_col(int l, int v) {
  return ((v / C) * LR + l) * C + v % C;
}

__device__ __forceinline__ float bf16_bits_f32(uint32_t b) { return __builtin_bit_cast(float, b << 16); }

// A row's logits.  Every load is made, of a column that exists where the lane
// has none: a load under a condition would be waited for at its end.
template <typename T, int LR, int V, int C>
struct RowLoad {
  uint32_t raw[sizeof(T) == 4 || C == 1 ? V : V / 2];
  __device__ __forceinline__ void load(const T* row, int E, int l) {
    if constexpr (C == 4) {
#pragma unroll
      for (int g = 0; g < V / 4; ++g) {
        const int c = min(balance_col<LR, 4>(l, 4 * g), E - 4);
        if constexpr (sizeof(T) == 4) {
          const u32x4 t = *reinterpret_cast<const u32x4*>(row + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) raw[4 * g + i] = t.v[i];
        } else {
          const uint2 t = *reinterpret_cast<const uint2*>(row + c);
          raw[2 * g] = t.x;
          raw[2 * g + 1] = t.y;
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = min(balance_col<LR, 1>(l, v), E - 1);
        if constexpr (sizeof(T) == 4) raw[v] = __builtin_bit_cast(uint32_t, row[c]);
        else raw[v] = row[c];
      }
    }
  }
  // As FP32; -inf beyond E and in a row that does not count, whatever it holds.
  __device__ __forceinline__ void values(float (&x)[V], int E, int l, bool on) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f;
      if constexpr (sizeof(T) == 4) f = __builtin_bit_cast(float, raw[v]);
      else if constexpr (C == 4) f = bf16_bits_f32((v & 1) ? raw[v / 2] >> 16 : raw[v / 2] & 0xFFFFu);
      else f = bf16_bits_f32(raw[v]);
      x[v] = (int)on & (int)(balance_col<LR, C>(l, v) < E) ? f : -__builtin_huge_valf();
    }
  }
};

// x becomes exp(x - max); `inv` the factor that makes probabilities of it;
// returns the log-sum-exp.  A row of -inf only: all three are 0.  A NaN or +inf
// anywhere makes every probability and the log-sum-exp NaN.  The sum lies in
// [1, E], so the instructions' reciprocal and logarithm (1 ulp) need no care
// for range.  A probability is within (|x - max| + 3) 2^-23 of itself, for the
// rounded product with log2 e and the reciprocal.  With the rounding's rest added
// and the reciprocal corrected (4096 tokens, FP32, against 64 bits) the losses were
// as far off as without (2.0e-8 and 2.8e-8 for two inputs), the gradient 8.9e-8 of
// its norm instead of 9.3e-8 (formed of FP32 torch operations 8.4e-8), and 65536
// tokens in bf16 took 26.3 us instead of 24.8.
template <int LR, int V>
__device__ __forceinline__ float row_softmax(float (&x)[V], float& inv) {
  float m = x[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
  m = row_max<LR>(m);
  m = m == -__builtin_huge_valf() ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    x[v] = __builtin_amdgcn_exp2f((x[v] - m) * 1.44269504f);
    s += x[v];
  }
  s = row_sum<LR>(s);
  inv = s == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(s);
  return s == 0.0f ? 0.0f : m + __builtin_amdgcn_logf(s) * 0.693147181f;
}

typedef float f32_quad __attribute__((ext_vector_type(4)));
typedef uint32_t u32_pair __attribute__((ext_vector_type(2)));

// Sum over the 64 lanes in a fixed order; every lane gets it.
template <typename A>
__device__ __forceinline__ A wave_sum(A v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// One part of group g: blocks of 8 wavefronts' rows, `parts` blocks apart.
// ALONE: there is no other (one group, one part), and losses, counts and tokens
// are written here (64 tokens of 128 experts 4.5 us in a graph).
template <typename T, int LR, int V, int C, bool ALONE>
__global__ __launch_bounds__(kBalThreads) void balance_parts_kernel(
    const T* __restrict__ logits, long long ld, const int32_t* __restrict__ ids, const uint8_t* __restrict__ valid,
    float* __restrict__ psum, int32_t* __restrict__ cnt, float* __restrict__ zpart, int32_t* __restrict__ npart,
    uint32_t* __restrict__ ticket, float* __restrict__ losses, int32_t* __restrict__ counts,
    int32_t* __restrict__ tokens, int S, int E, int k, int parts) {
  constexpr int RW = 64 / LR;                // rows a wavefront works on at a time
  constexpr int kCols = LR * V;
  __shared__ float sp[kBalWaves * kCols];
  __shared__ int32_t hist[kCols];
  __shared__ float sz[kBalWaves];
  __shared__ int32_t sn[kBalWaves];
  __shared__ double sd[kBalWaves];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l = lane % LR, rw = lane / LR;
  const int g = blockIdx.x / parts, part = blockIdx.x - g * parts;
  const long long base = (long long)g * S;
  const T* glogits = logits + base * ld;
  const int32_t* gids = ids + base * k;
  const uint32_t all = valid ? 0u : 1u;   // every token counts
  const uint8_t* gvalid = valid ? valid + base : reinterpret_cast<const uint8_t*>(gids);   // any byte: not looked at

  struct Rows {
    RowLoad<T, LR, V, C> r;
    uint32_t on;
    int id;   // this lane's slot of its row (l < k)
  } rows;
  auto request = [&](Rows& q, int t) {
    const int c = min(t, S - 1);
    q.r.load(glogits + (long long)c * ld, E, l);
    q.on = gvalid[c];
    q.id = gids[c * k + min(l, k - 1)];
  };
  auto count = [&](bool counted, int e) {
    if (counted & ((unsigned)e < (unsigned)E)) atomicAdd(&hist[e], 1);
  };
  // Round i of the part: the workgroups' blocks of one round lie side by side,
  // and the groups begin at different rounds; with a range of its own for each
  // part all of them read and wrote the same memory channels at a time (262144
  // tokens of 128 experts in 64 groups: both passes 96 against 90 us).
  constexpr int kStep = kBalWaves * RW;
  const int rounds = (S + parts * kStep - 1) / (parts * kStep);
  auto token = [&](int i) {
    int r = i + g % rounds;
    r -= r >= rounds ? rounds : 0;
    return (r * parts + part) * kStep + w * RW + rw;
  };
  request(rows, token(0));
  for (int i = tid; i < kCols; i += kBalThreads) hist[i] = 0;
  if (!ALONE && blockIdx.x == 0 && tid == 0) *ticket = 0;
  __syncthreads();

  if (k > LR) {   // slots that a row's lanes do not cover
    const int more = k - LR;
    for (int r = 0; r < rounds; ++r)
      for (int i = tid; i < kStep * more; i += kBalThreads) {
        const int t = (r * parts + part) * kStep + i / more, s = LR + i % more;
        if (t < S) count(!valid || gvalid[t], gids[t * k + s]);
      }
  }
  float P[V], zacc = 0.0f;
  int nacc = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) P[v] = 0.0f;
  for (int i = 0; i < rounds; ++i) {
    const int t = token(i);
    const bool now = (t < S) & ((rows.on | all) != 0u);   // no branch: a load waited for in one is waited for at its end
    float x[V], inv;
    rows.r.values(x, E, l, now);
    count(now & (l < k), rows.id);
    request(rows, token(min(i + 1, rounds - 1)));   // behind the last round: that one again
    __builtin_amdgcn_sched_barrier(0);              // before the work on this round, not after it
    const float z = row_softmax<LR, V>(x, inv);
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = __builtin_fmaf(x[v], inv, P[v]);
    zacc = __builtin_fmaf(z, z, zacc);
    nacc += now ? 1 : 0;
  }
  // the wavefront's row groups first (lanes l, l + LR, ...), then the wavefronts
  if constexpr (LR == 16) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      P[v] += __shfl_xor(P[v], 16);
      P[v] += __shfl_xor(P[v], 32);
    }
    zacc += __shfl_xor(zacc, 16);
    zacc += __shfl_xor(zacc, 32);
    nacc += __shfl_xor(nacc, 16);
    nacc += __shfl_xor(nacc, 32);
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
    if (rw == 0) sp[w * kCols + balance_col<LR, C>(l, v)] = P[v];
  if (lane == 0) {
    sz[w] = zacc;
    sn[w] = nacc;
  }
  __syncthreads();
  double dot = 0.0;
  for (int c = tid; c < E; c += kBalThreads) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kBalWaves; ++i) s += sp[i * kCols + c];
    if constexpr (ALONE) {
      counts[c] = hist[c];
      dot += (double)s * (double)hist[c];
    } else {
      psum[(size_t)blockIdx.x * E + c] = s;
      cnt[(size_t)blockIdx.x * E + c] = hist[c];
    }
  }
  if constexpr (ALONE) {
    dot = wave_sum(dot);
    if (lane == 0) sd[w] = dot;
    __syncthreads();
  }
  if (tid == 0) {
    float z = 0.0f;
    int n = 0;
    dot = 0.0;
#pragma unroll
    for (int i = 0; i < kBalWaves; ++i) {
      z += sz[i];
      n += sn[i];
      if (ALONE) dot += sd[i];
    }
    if constexpr (ALONE) {
      losses[0] = n > 0 ? (float)(dot * (double)E / ((double)k * (double)n * (double)n)) : 0.0f;
      losses[1] = n > 0 ? (float)((double)z / (double)n) : 0.0f;
      tokens[0] = tokens[1] = n;
    } else {
      zpart[blockIdx.x] = z;
      npart[blockIdx.x] = n;
    }
  }
}

// Second launch, one workgroup per (group, COLS experts): adds the parts, writes
// the group's counts, and leaves sum_e c_ge sum_t p_te in the workspace.  The
// workgroup that finishes last adds those up to the two losses; which one that
// is does not change the order of the sum.  32 experts a workgroup spread many
// parts over more workgroups; 128 make it one workgroup for one group, with
// nothing to wait for (128 parts of 128 experts: 4.2 against 6.8 us).
template <int COLS>
__global__ __launch_bounds__(kBalSumThreads) void balance_sum_kernel(
    const float* __restrict__ psum, const int32_t* __restrict__ cnt, const float* __restrict__ zpart,
    const int32_t* __restrict__ npart, double* __restrict__ dot, double* __restrict__ zsum,
    uint32_t* __restrict__ ticket, float* __restrict__ losses, int32_t* __restrict__ counts,
    int32_t* __restrict__ tokens, int E, int k, int G, int parts) {
  constexpr int kSlices = kBalSumThreads / COLS, kBatch = COLS == 32 ? 4 : 16;
  static_assert(COLS == 32 || COLS == 128);
  __shared__ double sd[kBalSumThreads];
  __shared__ int32_t si[kBalSumThreads];
  constexpr int kZWave = kBalSumWaves - 1;
  __shared__ double sdot[(COLS + 63) / 64];
  __shared__ double sz;
  __shared__ int32_t sn;
  __shared__ bool is_last;
  const int tid = threadIdx.x, splits = (E + COLS - 1) / COLS;
  const int g = blockIdx.x / splits, sp = blockIdx.x - g * splits;
  const int c = sp * COLS + tid % COLS, slice = tid / COLS;
  const float* gp = psum + (size_t)g * parts * E + min(c, E - 1);
  const int32_t* gc = cnt + (size_t)g * parts * E + min(c, E - 1);
  double p = 0.0;
  int n = 0;
  for (int i = slice; i < parts; i += kBatch * kSlices) {   // kBatch parts' loads at a time
    float a[kBatch];
    int b[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int j = min(i + u * kSlices, parts - 1);
      a[u] = gp[(size_t)j * E];
      b[u] = gc[(size_t)j * E];
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const bool in = i + u * kSlices < parts;
      p += in ? (double)a[u] : 0.0;
      n += in ? b[u] : 0;
    }
  }
  sd[tid] = p;
  si[tid] = n;
  double z = 0.0;   // the group's z and valid tokens: the last wavefront of its first workgroup
  int v = 0;
  if (sp == 0 && (tid >> 6) == kZWave)
    for (int i = tid & 63; i < parts; i += 64) {
      z += (double)zpart[(size_t)g * parts + i];
      v += npart[(size_t)g * parts + i];
    }
  __syncthreads();
  double d = 0.0;
  if (tid < COLS) {
    p = 0.0;
    n = 0;
#pragma unroll
    for (int s = 0; s < kSlices; ++s) {
      p += sd[s * COLS + tid];
      n += si[s * COLS + tid];
    }
    if (c < E) {
      counts[(size_t)g * E + c] = n;
      d = p * (double)n;
    }
  }
  if (tid < COLS || tid < 64) {
    d = wave_sum(d);
    if ((tid & 63) == 0) sdot[tid >> 6] = d;
  }
  if ((tid >> 6) == kZWave) {
    z = wave_sum(z);
    v = wave_sum(v);
    if ((tid & 63) == 0) {
      sz = z;
      sn = v;
    }
  }
  __syncthreads();
  d = sdot[0];
  if constexpr (COLS > 64) d += sdot[1];
  if (gridDim.x == 1) {
    if (tid == 0) {
      const double m = sn > 0 ? (double)sn : 1.0;
      losses[0] = (float)(d * (double)E / ((double)k * m * m));
      losses[1] = (float)(sz / m);
      tokens[0] = tokens[1] = sn;
    }
    return;
  }
  // one thread publishes what the last workgroup reads (agent scope: the workgroups run on different XCDs)
  if (tid == 0) {
    __hip_atomic_store(&dot[blockIdx.x], d, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (sp == 0) {
      __hip_atomic_store(&zsum[g], sz, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&tokens[g], sn, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    is_last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!is_last) return;
  double bal = 0.0;
  int N = 0;
  z = 0.0;
  for (int i = tid; i < G; i += kBalSumThreads) {
    const int m = __hip_atomic_load(&tokens[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    double s = 0.0;
    for (int j = 0; j < splits; ++j)
      s += __hip_atomic_load(&dot[(size_t)i * splits + j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (m > 0) bal += s * (double)E / ((double)k * (double)m * (double)m);
    z += __hip_atomic_load(&zsum[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    N += m;
  }
  bal = wave_sum(bal);
  z = wave_sum(z);
  N = wave_sum(N);
  if ((tid & 63) == 0) {
    sd[tid >> 6] = bal;
    sd[kBalSumWaves + (tid >> 6)] = z;
    si[tid >> 6] = N;
  }
  __syncthreads();
  if (tid == 0) {
#pragma unroll
    for (int i = 1; i < kBalSumWaves; ++i) {
      bal += sd[i];
      z += sd[kBalSumWaves + i];
      N += si[i];
    }
    losses[0] = (float)(bal / (double)G);
    losses[1] = N > 0 ? (float)(z / (double)N) : 0.0f;
    tokens[G] = N;
  }
}

// The gradient of one part's rows: p_e (F_e - sum_j F_j p_j + zc logsumexp), with
// F and zc the factors that do not change from row to row of a group.  262144
// tokens of 128 experts, FP32: 41 us behind the forward pass, 268 MB (6.5 TB/s,
// part of the logits coming from the memory-side cache).
template <typename T, int LR, int V, int C>
__global__ __launch_bounds__(kBalThreads) void balance_backward_kernel(
    const T* __restrict__ logits, long long ld, const uint8_t* __restrict__ valid, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ tokens, const float* __restrict__ grad_losses, T* __restrict__ dlogits, long long ld_d,
    int S, int E, int k, int G, int parts) {
  constexpr int RW = 64 / LR;
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l = lane % LR, rw = lane / LR;
  const int g = blockIdx.x / parts, part = blockIdx.x - g * parts;
  const long long base = (long long)g * S;
  struct Rows {
    RowLoad<T, LR, V, C> r;
    uint32_t on;
  } rows;
  const uint32_t all = valid ? 0u : 1u;   // every token counts
  const uint8_t* gvalid = valid ? valid + base : reinterpret_cast<const uint8_t*>(logits);   // any byte: not looked at
  auto request = [&](Rows& q, int t) {
    const int c = min(t, S - 1);
    q.r.load(logits + (base + c) * ld, E, l);
    q.on = gvalid[valid ? c : 0];
  };
  // The forward pass's rounds, the last first: their rows are what the
  // memory-side cache still holds of the logits, and the gradient is written
  // past the caches, as streaming data, so that it stays so (262144 tokens of
  // 128 experts, both passes 89 us, with such stores 79, and in this order 73).
  constexpr int kStep = kBalWaves * RW;
  const int rounds = (S + parts * kStep - 1) / (parts * kStep);
  auto token = [&](int i) {
    int r = rounds - 1 - i + g % rounds;
    r -= r >= rounds ? rounds : 0;
    return (r * parts + part) * kStep + w * RW + rw;
  };
  request(rows, token(0));
  const float n = (float)max(tokens[g], 1), N = (float)max(tokens[G], 1);
  const float fb = grad_losses[0] * ((float)E / ((float)G * (float)k * n * n));
  const float zc = grad_losses[1] * (2.0f / N);
  float F[V];   // grad_losses[0] / (G n_g) * f_ge
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = balance_col<LR, C>(l, v);
    F[v] = (float)counts[(size_t)g * E + min(c, E - 1)];
  }
#pragma unroll
  for (int v = 0; v < V; ++v) F[v] = balance_col<LR, C>(l, v) < E ? fb * F[v] : 0.0f;
  for (int i = 0; i < rounds; ++i) {
    const int t = token(i);
    const bool in = t < S, now = in & ((rows.on | all) != 0u);
    float x[V], inv;
    rows.r.values(x, E, l, now);
    request(rows, token(min(i + 1, rounds - 1)));   // behind the last round: that one again
    __builtin_amdgcn_sched_barrier(0);              // before the work on this round, not after it
    const float z = row_softmax<LR, V>(x, inv);
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) dot = __builtin_fmaf(x[v], F[v], dot);
    dot = row_sum<LR>(dot) * inv;
    const float zt = zc * z - dot;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = now ? x[v] * inv * (F[v] + zt) : 0.0f;
    if (!in) continue;
    T* out = dlogits + (base + t) * ld_d;
    if constexpr (C == 4) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const int c = balance_col<LR, 4>(l, 4 * q);
        if (c >= E) continue;
        if constexpr (sizeof(T) == 4) {
          __builtin_nontemporal_store(f32_quad{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]},
                                      reinterpret_cast<f32_quad*>(out + c));
        } else {
          __builtin_nontemporal_store(u32_pair{f32_to_bf16_rne(x[4 * q]) | (uint32_t)f32_to_bf16_rne(x[4 * q + 1]) << 16,
                                               f32_to_bf16_rne(x[4 * q + 2]) | (uint32_t)f32_to_bf16_rne(x[4 * q + 3]) << 16},
                                      reinterpret_cast<u32_pair*>(out + c));
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = balance_col<LR, 1>(l, v);
        if (c < E) {
          if constexpr (sizeof(T) == 4) out[c] = x[v];
          else out[c] = f32_to_bf16_rne(x[v]);
        }
      }
    }
  }
}

}  // namespace moe
