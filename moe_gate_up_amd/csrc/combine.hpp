// The experts' rows back to their tokens, and the gradients (the definitions are
// at moe_decode_combine in include/moe_decode.h).
#pragma once

#include "pieces.hpp"

namespace moe {

constexpr int kCombineThreads = 256;
constexpr int kCombineMaxK = 64;

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
  const int left = a.N - c;
  const int32_t* at = a.positions + (long long)t * a.k;
  float sum[kPiece];
  if (add) {
    Piece<T> p;
    p.load(add + (long long)t * a.ld_add + c, left);
    p.values(sum);
  } else {
#pragma unroll
    for (int i = 0; i < kPiece; ++i) sum[i] = 0.0f;
  }
  for (int j = 0; j < a.k; ++j) {
    const int m = at[j];
    if ((unsigned)m >= (unsigned)a.M) continue;   // uniform: one token a workgroup
    const float w = a.weights ? a.weights[(long long)t * a.k + j] : 1.0f;
    Piece<T> p;
    p.load(rows + (long long)m * a.ld_rows + c, left);
    float f[kPiece];
    p.values(f);
#pragma unroll
    for (int i = 0; i < kPiece; ++i) sum[i] = __builtin_fmaf(w, f[i], sum[i]);
  }
  Piece<T> p;
  p.set(sum);
  p.store(y + (long long)t * a.ld_y + c, left);
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
      const int left = a.N - c;
      Piece<T> p;
      float g[kPiece];
      p.load(dy + (long long)t * a.ld_dy + c, left);
      p.values(g);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const int m = j0 + j < a.k ? at[j0 + j] : -1;
        if ((unsigned)m >= (unsigned)a.M) continue;
        float f[kPiece];
        if (a.dweights) {
          p.load(rows + (long long)m * a.ld_rows + c, left);
          p.values(f);
#pragma unroll
          for (int i = 0; i < kPiece; ++i) dot[j] = __builtin_fmaf(f[i], g[i], dot[j]);
        }
        const float wt = a.weights ? a.weights[(long long)t * a.k + j0 + j] : 1.0f;
#pragma unroll
        for (int i = 0; i < kPiece; ++i) f[i] = wt * g[i];
        p.set(f);
        p.store(drows + (long long)m * a.ld_d + c, left);
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
