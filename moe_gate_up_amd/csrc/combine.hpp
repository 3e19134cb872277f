// The experts' rows back to their tokens, and the gradients (the definitions are
// at moe_decode_combine in include/moe_decode.h).
//
// Memory bounds both: every row is read (and its gradient written) once.  One token a
// workgroup, so that positions and weights are the workgroup's, and the rows of several
// slots requested together.  4096 tokens, a fifth of them padding, 8 rows of 2048 bf16:
// forward 28 us for 141 MB (5.1 TB/s; 8 rows together, whose registers leave fewer
// wavefronts, 31; each row waited for 37), backward 40 us for 231 MB (5.8 TB/s; 4
// together 47, through the caches 41).  A slot without a row must not ask all for the same
// one instead: with row 0 for padding the forward pass took 34.
#pragma once

#include "pieces.hpp"

namespace moe {

constexpr int kCombineThreads = 256;
constexpr int kCombineMaxK = 64;
constexpr int kCombineSlots = 4;

struct CombineArgs {
  const int32_t* positions;
  const float* weights;   // nullptr: 1
  long long ld_rows, ld_add, ld_y;
  int M, T, N, k;
  int chunks;             // workgroups of one token
};

// One piece of 8 columns of one token a thread.
template <typename T>
__global__ __launch_bounds__(kCombineThreads) void combine_kernel(const T* __restrict__ rows, const T* add, T* y,
                                                                  CombineArgs a) {
  const int t = (int)blockIdx.x / a.chunks;
  const int c = (((int)blockIdx.x - t * a.chunks) * (int)blockDim.x + (int)threadIdx.x) * kPiece;
  if (c >= a.N) return;
  const int32_t* at = a.positions + (long long)t * a.k;
  // kCombineSlots rows at a time, all requested before the first is used; a slot without a row asks for another slot's
  // and does not use it
  Piece<T> base, p[kCombineSlots];
  float sum[kPiece];
#pragma unroll
  for (int i = 0; i < kPiece; ++i) sum[i] = 0.0f;
  if (add) base.request(add + (long long)t * a.ld_add, c, a.N);
  for (int j0 = 0; j0 < a.k; j0 += kCombineSlots) {
    int m[kCombineSlots];
    float w[kCombineSlots];
#pragma unroll
    for (int j = 0; j < kCombineSlots; ++j) {
      m[j] = at[min(j0 + j, a.k - 1)];
      m[j] = j0 + j < a.k && (unsigned)m[j] < (unsigned)a.M ? m[j] : -1;
      w[j] = a.weights ? a.weights[(long long)t * a.k + min(j0 + j, a.k - 1)] : 1.0f;
    }
    int some = m[0];
#pragma unroll
    for (int j = 1; j < kCombineSlots; ++j) some = max(some, m[j]);
    if (some < 0) continue;   // uniform: one token a workgroup
#pragma unroll
    for (int j = 0; j < kCombineSlots; ++j) p[j].request(rows + (m[j] < 0 ? some : m[j]) * a.ld_rows, c, a.N);
#pragma unroll
    for (int j = 0; j < kCombineSlots; ++j) {
      if (m[j] < 0) continue;
      p[j].settle(c, a.N);
      float f[kPiece];
      p[j].values(f);
#pragma unroll
      for (int i = 0; i < kPiece; ++i) sum[i] = __builtin_fmaf(w[j], f[i], sum[i]);
    }
  }
  if (add) {
    float f[kPiece];
    base.settle(c, a.N, add == y ? add + (long long)t * a.ld_add : nullptr);
    base.values(f);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) sum[i] += f[i];
  }
  Piece<T> out;
  out.set(sum);
  out.stream(y + (long long)t * a.ld_y, c, a.N);
}

struct CombineBackwardArgs {
  const int32_t* positions;
  const float* weights;
  float* dweights;        // nullptr: not asked for
  long long ld_dy, ld_rows, ld_d;
  int M, T, N, k;
};

// One token a workgroup, its columns in turns; 8 slots at a time.
template <typename T>
__global__ __launch_bounds__(kCombineThreads) void combine_backward_kernel(const T* __restrict__ dy,
                                                                           const T* __restrict__ rows,
                                                                           T* __restrict__ drows, CombineBackwardArgs a) {
  constexpr int J = 8;
  __shared__ float part[kCombineThreads / 64][J];
  const int t = (int)blockIdx.x, tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int32_t* at = a.positions + (long long)t * a.k;
  for (int j0 = 0; j0 < a.k; j0 += J) {
    float dot[J];
#pragma unroll
    for (int j = 0; j < J; ++j) dot[j] = 0.0f;
    for (int c = tid * kPiece; c < a.N; c += (int)blockDim.x * kPiece) {
      Piece<T> p;
      float g[kPiece];
      int m[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        m[j] = at[min(j0 + j, a.k - 1)];
        m[j] = j0 + j < a.k && (unsigned)m[j] < (unsigned)a.M ? m[j] : -1;
      }
      int some = m[0];
#pragma unroll
      for (int j = 1; j < J; ++j) some = max(some, m[j]);
      if (some < 0) break;   // uniform: one token a workgroup
      p.request(dy + (long long)t * a.ld_dy, c, a.N);
      Piece<T> q[J];
      if (a.dweights) {
#pragma unroll
        for (int j = 0; j < J; ++j) q[j].request(rows + (m[j] < 0 ? some : m[j]) * a.ld_rows, c, a.N);
      }
      p.settle(c, a.N);
      p.values(g);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (m[j] < 0) continue;
        float f[kPiece];
        if (a.dweights) {
          q[j].settle(c, a.N);
          q[j].values(f);
#pragma unroll
          for (int i = 0; i < kPiece; ++i) dot[j] = __builtin_fmaf(f[i], g[i], dot[j]);
        }
        const float wt = a.weights ? a.weights[(long long)t * a.k + j0 + j] : 1.0f;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) f[i] = wt * g[i];
        Piece<T> o;
        o.set(f);
        o.stream(drows + m[j] * a.ld_d, c, a.N);
      }
    }
    if (!a.dweights) continue;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float s = wave_sum_row3(dot[j]);
      if (lane == 63) part[w][j] = s;
    }
    __syncthreads();
    if (tid < J && j0 + tid < a.k) {
      float s = 0.0f;
      for (int i = 0; i < (int)blockDim.x / 64; ++i) s += part[i][tid];
      const bool on = (unsigned)at[j0 + tid] < (unsigned)a.M;
      a.dweights[(long long)t * a.k + j0 + tid] = on ? s : 0.0f;
    }
    __syncthreads();
  }
}

}  // namespace moe
