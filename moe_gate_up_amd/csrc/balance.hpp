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
// Forward: a workgroup takes a contiguous part of one group's tokens; each
// lane adds up its columns' probabilities over its rows, the wavefronts' sums
// are added in LDS in a fixed order, and the slots are counted with integer
// LDS atomics, whose order cannot change the result.  The parts' sums go to
// the workspace, and a second launch adds them (FP64, fixed order).
// Backward: the same walk with f_ge in registers; the softmax is computed
// again rather than stored (a stored one would be T E more bytes each way).
#pragma once

#include "prims.hpp"
#include "router.hpp"

namespace moe {

constexpr int kBalThreads = 512;
constexpr int kBalWaves = kBalThreads / 64;
constexpr int kBalMaxExperts = 1024;
constexpr int kBalMaxK = 64;
constexpr int kBalSumThreads = 256;
constexpr int kBalSumCols = 32;       // experts one workgroup of the second launch adds up
constexpr int kBalTargetParts = 512;  // workgroups of a pass: 2 per CU

// Parts each group's tokens are cut into: enough workgroups for the chip, at
// least 32 tokens each.
__host__ __device__ constexpr int balance_parts(int S, int G) {
  const int by_chip = (kBalTargetParts + G - 1) / G;
  const int by_work = (S + 31) / 32;
  return by_chip < by_work ? by_chip : (by_work < 1 ? 1 : by_work);
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

// A row's logits as FP32, -inf beyond E.
template <typename T, int LR, int V, int C>
struct RowLoad {
  uint32_t raw[sizeof(T) == 4 || C == 1 ? V : V / 2];
  __device__ __forceinline__ void load(const T* row, int E, int l) {
    if constexpr (C == 4) {
#pragma unroll
      for (int g = 0; g < V / 4; ++g) {
        const int c = balance_col<LR, 4>(l, 4 * g);
        if constexpr (sizeof(T) == 4) {
          u32x4 t{{0, 0, 0, 0}};
          if (c < E) t = *reinterpret_cast<const u32x4*>(row + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) raw[4 * g + i] = t.v[i];
        } else {
          uint2 t{0, 0};
          if (c < E) t = *reinterpret_cast<const uint2*>(row + c);
          raw[2 * g] = t.x;
          raw[2 * g + 1] = t.y;
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = balance_col<LR, 1>(l, v);
        raw[v] = 0;
        if (c < E) {
          if constexpr (sizeof(T) == 4) raw[v] = __builtin_bit_cast(uint32_t, row[c]);
          else raw[v] = row[c];
        }
      }
    }
  }
  __device__ __forceinline__ void values(float (&x)[V], int E, int l) const {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f;
      if constexpr (sizeof(T) == 4) f = __builtin_bit_cast(float, raw[v]);
      else if constexpr (C == 4) f = bf16_bits_f32((v & 1) ? raw[v / 2] >> 16 : raw[v / 2] & 0xFFFFu);
      else f = bf16_bits_f32(raw[v]);
      x[v] = balance_col<LR, C>(l, v) < E ? f : -__builtin_huge_valf();
    }
  }
};

// x becomes the row's probabilities; returns its log-sum-exp.  A row of -inf
// only: probabilities and log-sum-exp 0.  A NaN or +inf anywhere makes every
// probability and the log-sum-exp NaN.
template <int LR, int V>
__device__ __forceinline__ float row_softmax(float (&x)[V]) {
  float m = x[0];
#pragma unroll
  for (int v = 1; v < V; ++v) m = fmaxf(m, x[v]);
  m = row_max<LR>(m);
  m = m == -__builtin_huge_valf() ? 0.0f : m;
  float s = 0.0f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    x[v] = __expf(x[v] - m);
    s += x[v];
  }
  s = row_sum<LR>(s);
  const float inv = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
  for (int v = 0; v < V; ++v) x[v] *= inv;
  return s == 0.0f ? 0.0f : m + __logf(s);
}

// One part: tokens [first, last) of group g.
template <typename T, int LR, int V, int C>
__global__ __launch_bounds__(kBalThreads) void balance_parts_kernel(
    const T* __restrict__ logits, long long ld, const int32_t* __restrict__ ids, const uint8_t* __restrict__ valid,
    float* __restrict__ psum, int32_t* __restrict__ cnt, float* __restrict__ zpart, int32_t* __restrict__ npart,
    uint32_t* __restrict__ ticket, int S, int E, int k, int parts) {
  constexpr int RW = 64 / LR;                // rows a wavefront works on at a time
  constexpr int kCols = LR * V;
  __shared__ float sp[kBalWaves * kCols];
  __shared__ int32_t hist[kCols];
  __shared__ float sz[kBalWaves * RW];
  __shared__ int32_t sn[kBalWaves * RW];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int l = lane % LR, rw = lane / LR;
  const int g = blockIdx.x / parts, part = blockIdx.x - g * parts;
  const int per = (S + parts - 1) / parts;
  const int first = min(part * per, S), last = min(first + per, S);
  const long long base = (long long)g * S;
  for (int i = tid; i < kCols; i += kBalThreads) hist[i] = 0;
  if (blockIdx.x == 0 && tid == 0) *ticket = 0;
  __syncthreads();

  // slots of valid tokens
  const int32_t* gids = ids + base * k;
  for (int i = first * k + tid; i < last * k; i += kBalThreads) {
    const bool on = !valid || valid[base + i / k];
    const int e = gids[i];
    if (on && (unsigned)e < (unsigned)E) atomicAdd(&hist[e], 1);
  }

  float P[V], zacc = 0.0f;
  int nacc = 0;
#pragma unroll
  for (int v = 0; v < V; ++v) P[v] = 0.0f;
  for (int t0 = first; t0 < last; t0 += kBalWaves * RW) {
    const int t = t0 + w * RW + rw;
    const bool on = t < last && (!valid || valid[base + t]);
    RowLoad<T, LR, V, C> r;
    r.load(logits + (base + min(t, last - 1)) * ld, E, l);
    float x[V];
    r.values(x, E, l);
    const float z = row_softmax<LR, V>(x);
    // selects, not products: an invalid row may hold NaN
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] += on ? x[v] : 0.0f;
    zacc += on ? z * z : 0.0f;
    nacc += on ? 1 : 0;
  }
  // the wavefront's row groups first (lanes l, l + LR, ...), then the wavefronts
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if constexpr (LR == 16) {
      P[v] += __shfl_xor(P[v], 16);
      P[v] += __shfl_xor(P[v], 32);
    }
    if (rw == 0) sp[w * kCols + balance_col<LR, C>(l, v)] = P[v];
  }
  if (l == 0) {
    sz[w * RW + rw] = zacc;
    sn[w * RW + rw] = nacc;
  }
  __syncthreads();
  for (int c = tid; c < E; c += kBalThreads) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kBalWaves; ++i) s += sp[i * kCols + c];
    psum[(size_t)blockIdx.x * E + c] = s;
    cnt[(size_t)blockIdx.x * E + c] = hist[c];
  }
  if (tid == 0) {
    float z = 0.0f;
    int n = 0;
    for (int i = 0; i < kBalWaves * RW; ++i) {
      z += sz[i];
      n += sn[i];
    }
    zpart[blockIdx.x] = z;
    npart[blockIdx.x] = n;
  }
}

// Sum over the workgroup in a fixed order; every thread gets it.
template <int THREADS, typename A>
__device__ __forceinline__ A block_sum(A v, A* scratch, int tid) {
  scratch[tid] = v;
  __syncthreads();
#pragma unroll
  for (int o = THREADS / 2; o > 0; o >>= 1) {
    if (tid < o) scratch[tid] += scratch[tid + o];
    __syncthreads();
  }
  const A s = scratch[0];
  __syncthreads();
  return s;
}

// Second launch, one workgroup per (group, 32 experts): adds the parts, writes
// the group's counts, and leaves sum_e c_ge sum_t p_te in the workspace.  The
// workgroup that finishes last adds those up to the two losses; which one that
// is does not change the order of the sum.
__global__ __launch_bounds__(kBalSumThreads) void balance_sum_kernel(
    const float* __restrict__ psum, const int32_t* __restrict__ cnt, const float* __restrict__ zpart,
    const int32_t* __restrict__ npart, double* __restrict__ dot, double* __restrict__ zsum,
    uint32_t* __restrict__ ticket, float* __restrict__ losses, int32_t* __restrict__ counts,
    int32_t* __restrict__ tokens, int E, int k, int G, int parts) {
  constexpr int kSlices = kBalSumThreads / kBalSumCols;
  __shared__ double sd[kBalSumThreads];
  __shared__ int32_t si[kBalSumThreads];
  __shared__ bool is_last;
  const int tid = threadIdx.x, splits = balance_splits(E);
  const int g = blockIdx.x / splits, sp = blockIdx.x - g * splits;
  const int c = sp * kBalSumCols + tid % kBalSumCols, slice = tid / kBalSumCols;
  double p = 0.0;
  int n = 0;
  if (c < E)
    for (int i = slice; i < parts; i += kSlices) {
      p += (double)psum[((size_t)g * parts + i) * E + c];
      n += cnt[((size_t)g * parts + i) * E + c];
    }
  sd[tid] = p;
  si[tid] = n;
  __syncthreads();
  p = 0.0;
  n = 0;
  if (tid < kBalSumCols) {
    for (int s = 0; s < kSlices; ++s) {
      p += sd[s * kBalSumCols + tid];
      n += si[s * kBalSumCols + tid];
    }
    if (c < E) counts[(size_t)g * E + c] = n;
  }
  __syncthreads();
  const double d = block_sum<kBalSumThreads>(tid < kBalSumCols ? p * (double)n : 0.0, sd, tid);
  if (sp == 0) {
    double z = 0.0;
    int v = 0;
    for (int i = tid; i < parts; i += kBalSumThreads) {
      z += (double)zpart[(size_t)g * parts + i];
      v += npart[(size_t)g * parts + i];
    }
    z = block_sum<kBalSumThreads>(z, sd, tid);
    v = block_sum<kBalSumThreads>(v, si, tid);
    if (tid == 0) {
      zsum[g] = z;
      tokens[g] = v;
    }
  }
  if (tid == 0) {
    dot[blockIdx.x] = d;
    __threadfence();
    is_last = __hip_atomic_fetch_add(ticket, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
  }
  __syncthreads();
  if (!is_last) return;
  __threadfence();
  double bal = 0.0, z = 0.0;
  int N = 0;
  for (int i = tid; i < G; i += kBalSumThreads) {
    const int v = __hip_atomic_load(&tokens[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    double s = 0.0;
    for (int j = 0; j < splits; ++j)
      s += __hip_atomic_load(&dot[(size_t)i * splits + j], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (v > 0) bal += s * (double)E / ((double)k * (double)v * (double)v);
    z += __hip_atomic_load(&zsum[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    N += v;
  }
  bal = block_sum<kBalSumThreads>(bal, sd, tid);
  z = block_sum<kBalSumThreads>(z, sd, tid);
  N = block_sum<kBalSumThreads>(N, si, tid);
  if (tid == 0) {
    losses[0] = (float)(bal / (double)G);
    losses[1] = N > 0 ? (float)(z / (double)N) : 0.0f;
    tokens[G] = N;
  }
}

template <typename T, int LR, int V, int C>
__global__ __launch_bounds__(kBalThreads) void balance_backward_kernel(
    const T* __restrict__ logits, long long ld, const uint8_t* __restrict__ valid, const int32_t* __restrict__ counts,
    const int32_t* __restrict__ tokens, const float* __restrict__ grad_losses, T* __restrict__ dlogits, long long ld_d,
    int S, int E, int k, int G, int parts) {
  constexpr int RW = 64 / LR;
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int l = lane % LR, rw = lane / LR;
  const int g = blockIdx.x / parts, part = blockIdx.x - g * parts;
  const int per = (S + parts - 1) / parts;
  const int first = min(part * per, S), last = min(first + per, S);
  const long long base = (long long)g * S;
  const float n = (float)max(tokens[g], 1), N = (float)max(tokens[G], 1);
  const float fb = grad_losses[0] * ((float)E / ((float)G * (float)k * n * n));
  const float zc = grad_losses[1] * (2.0f / N);
  float F[V];   // grad_losses[0] / (G n_g) * f_ge
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = balance_col<LR, C>(l, v);
    F[v] = c < E ? fb * (float)counts[(size_t)g * E + c] : 0.0f;
  }
  for (int t0 = first; t0 < last; t0 += kBalWaves * RW) {
    const int t = t0 + w * RW + rw;
    const bool in = t < last;
    const bool on = in && (!valid || valid[base + t]);
    RowLoad<T, LR, V, C> r;
    r.load(logits + (base + min(t, last - 1)) * ld, E, l);
    float x[V];
    r.values(x, E, l);
    const float z = row_softmax<LR, V>(x);
    float dot = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) dot += x[v] * F[v];
    dot = row_sum<LR>(dot);
    const float zt = zc * z - dot;
#pragma unroll
    for (int v = 0; v < V; ++v) x[v] = on ? x[v] * (F[v] + zt) : 0.0f;
    if (!in) continue;
    T* out = dlogits + (base + t) * ld_d;
    if constexpr (C == 4) {
#pragma unroll
      for (int q = 0; q < V / 4; ++q) {
        const int c = balance_col<LR, 4>(l, 4 * q);
        if (c >= E) continue;
        if constexpr (sizeof(T) == 4) {
          *reinterpret_cast<float4*>(out + c) = float4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
        } else {
          *reinterpret_cast<uint2*>(out + c) =
              uint2{f32_to_bf16_rne(x[4 * q]) | (uint32_t)f32_to_bf16_rne(x[4 * q + 1]) << 16,
                    f32_to_bf16_rne(x[4 * q + 2]) | (uint32_t)f32_to_bf16_rne(x[4 * q + 3]) << 16};
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
