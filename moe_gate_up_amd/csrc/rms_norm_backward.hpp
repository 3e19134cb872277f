// Gradients of the root-mean-square norm (the definition is at
// moe_decode_rms_norm_backward in include/moe_decode.h).
//
// A workgroup of 16 wavefronts holds 16 / WR rows at a time, each in the registers of
// WR of them, P pieces of 8 columns a lane, and keeps its sum for dweight in registers
// over its rows.  The next row's inputs are requested before the present one is worked
// on.  The wavefronts' sums for dweight are halved pairwise in LDS, the workgroups' are
// added by a second launch.
//
// Memory bounds it: 16384 x 2048 bf16 with dsum 50 us for 268 MB (5.4 TB/s; a copy
// 6.3), and 5 for the second launch.  One piece a lane and one workgroup a CU: four pieces,
// so that a wavefront holds a row, spill (159 us, and 92 at 8 wavefronts a CU).
#pragma once

#include "rms_norm.hpp"

namespace moe {

constexpr int kNormBackThreads = 1024;
constexpr int kNormBackWaves = kNormBackThreads / 64;
constexpr int kNormBackParts = 256;   // workgroups, one a CU: what a CU holds of them

struct NormBackwardArgs {
  long long ld_dy, ld_r, ld_dsum, ld_dx;
  const float* rstd;
  float* part;   // [workgroups, H]: each one's sum of dy r rstd over its rows
  int M, H;
};

// Row group i of workgroup b takes rows b + gridDim.x * (i + n * the number of groups).
template <typename T, typename W, int WR, int P>
__global__ __launch_bounds__(kNormBackThreads) void rms_norm_backward_kernel(const T* __restrict__ dy,
                                                                             const T* __restrict__ r,
                                                                             const W* __restrict__ weight, const T* dsum,
                                                                             T* dx, NormBackwardArgs a) {
  constexpr int R = kNormBackWaves / WR;   // rows at a time
  constexpr int kRow = 64 * WR * P * kPiece;
  __shared__ float lds[R > 1 ? R / 2 * kRow : 1];
  __shared__ float sums[2][kNormBackWaves];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int group = w / WR, l = (w % WR) * 64 + lane;
  float dw[P][kPiece];
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < kPiece; ++j) dw[i][j] = 0.0f;
  auto column = [&](int i) { return (i * 64 * WR + l) * kPiece; };
  Piece<W> pw[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    pw[i].request(weight, column(i), a.H);
    pw[i].settle(column(i), a.H);
  }
  Piece<T> pr[P], pg[P], ps[P];
  float rstd = 0.0f;
  // the row after the last one is requested too: that one again
  auto request = [&](long long m) {
    m = m < a.M ? m : a.M - 1;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      pr[i].request(r + m * a.ld_r, column(i), a.H);
      pg[i].request(dy + m * a.ld_dy, column(i), a.H);
      if (dsum) ps[i].request(dsum + m * a.ld_dsum, column(i), a.H);
    }
    rstd = a.rstd[m];
  };
  const long long step = (long long)gridDim.x * R;
  constexpr bool AHEAD = P == 1;   // longer pieces need the registers
  if (AHEAD) request(blockIdx.x + (long long)gridDim.x * group);
  int turn = 0;
  for (long long m0 = blockIdx.x; m0 < a.M; m0 += step, turn ^= 1) {
    const long long m = m0 + (long long)gridDim.x * group;
    const bool on = m < a.M;   // of all of a row's wavefronts; the others come to the barrier as well
    if (!AHEAD) request(m);
    float n[P][kPiece], g[P][kPiece], t[P][kPiece], dot = 0.0f;
    const float rs = rstd;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      pr[i].settle(column(i), a.H);
      pg[i].settle(column(i), a.H);
      pr[i].values(n[i]);
      pg[i].values(g[i]);
      if (dsum) {
        ps[i].settle(column(i), a.H, dsum == dx ? dsum + (on ? m : a.M - 1) * a.ld_dsum : nullptr);
        ps[i].values(t[i]);
      } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j) t[i][j] = 0.0f;
      }
    }
    if (AHEAD) {
      request(m + step);
      __builtin_amdgcn_sched_barrier(0);   // before the work on this row
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float wt[kPiece];
      pw[i].values(wt);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        n[i][j] *= rs;
        if (on) dw[i][j] = __builtin_fmaf(g[i][j], n[i][j], dw[i][j]);
        g[i][j] *= wt[j];
        dot = __builtin_fmaf(g[i][j], n[i][j], dot);
      }
    }
    dot = wave_sum_f32(dot);
    if constexpr (WR > 1) {   // two places in turn: a sum is read before its place is written again
      if (lane == 0) sums[turn][w] = dot;
      __syncthreads();
      dot = 0.0f;
#pragma unroll
      for (int i = 0; i < WR; ++i) dot += sums[turn][group * WR + i];
    }
    if (!on) continue;
    const float mean = dot / (float)a.H;
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
      for (int j = 0; j < kPiece; ++j) t[i][j] = __builtin_fmaf(rs, g[i][j] - n[i][j] * mean, t[i][j]);
      Piece<T> o;
      o.set(t[i]);
      o.stream(dx + m * a.ld_dx, column(i), a.H);
    }
  }
  // the upper half of the groups' sums onto the lower half's, until one is left
#pragma unroll
  for (int half = R / 2; half > 0; half /= 2) {
    if (group >= half && group < 2 * half)
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < kPiece; ++j) lds[(group - half) * kRow + (i * kPiece + j) * 64 * WR + l] = dw[i][j];
    __syncthreads();
    if (group < half)
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < kPiece; ++j) dw[i][j] += lds[group * kRow + (i * kPiece + j) * 64 * WR + l];
    __syncthreads();
  }
  if (group > 0) return;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    Piece<float> o;
    o.set(dw[i]);
    o.store(a.part + (long long)blockIdx.x * a.H, column(i), a.H);
  }
}

// dweight: the workgroups' sums added in FP64 in a fixed order, 32 columns a
// workgroup, 32 of the sums' rows at a time, 8 of each thread's requested together.
constexpr int kNormSumThreads = 1024;
__global__ __launch_bounds__(kNormSumThreads) void rms_norm_weight_kernel(const float* __restrict__ part,
                                                                          float* __restrict__ dweight, int rows, int H) {
  __shared__ double lds[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = (int)blockIdx.x * 32 + c;
  double s = 0.0;
  if (col < H) {
    float v[kNormBackParts / 32];
#pragma unroll
    for (int i = 0; i < kNormBackParts / 32; ++i) v[i] = part[(long long)min(g + 32 * i, rows - 1) * H + col];
#pragma unroll
    for (int i = 0; i < kNormBackParts / 32; ++i) s += g + 32 * i < rows ? (double)v[i] : 0.0;
  }
  lds[g][c] = s;
  __syncthreads();
  if (g == 0 && col < H) {
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < 32; ++i) v += lds[i][c];
    dweight[col] = (float)v;
  }
}

}  // namespace moe
