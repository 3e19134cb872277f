// Gradients of the root-mean-square norm (the definition is at
// moe_decode_rms_norm_backward in include/moe_decode.h).
//
// A row lies in the registers as in the forward pass.  A workgroup walks over rows
// and keeps its sum for dweight in registers; the workgroups' sums are added by a
// second launch.
#pragma once

#include "rms_norm.hpp"

namespace moe {

struct NormBackwardArgs {
  long long ld_dy, ld_r, ld_dsum, ld_dx;
  const float* rstd;
  float* part;   // [workgroups, H]: each one's sum of dy r rstd over its rows
  int M, H;
};

// The rows of a workgroup lie gridDim.x (times its rows) apart.
template <typename T, typename W, int WR, int P>
__global__ __launch_bounds__(norm_threads(WR)) void rms_norm_backward_kernel(const T* __restrict__ dy,
                                                                             const T* __restrict__ r,
                                                                             const W* __restrict__ weight, const T* dsum,
                                                                             T* dx, NormBackwardArgs a) {
  constexpr int R = norm_rows(WR);
  __shared__ double lds[WR == 1 ? 1 : WR];
  __shared__ float join[WR == 1 ? 3 : 1][WR == 1 ? 64 * P * kPiece : 1];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int l = WR == 1 ? lane : (int)threadIdx.x;
  float dw[P][kPiece];
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < kPiece; ++j) dw[i][j] = 0.0f;
  for (int m = (int)blockIdx.x * R + (WR == 1 ? w : 0); m < a.M; m += (int)gridDim.x * R) {
    Piece<T> pr[P], pg[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = (i * 64 * WR + l) * kPiece, left = a.H - c;
      pr[i].load(r + (long long)m * a.ld_r + c, left);
      pg[i].load(dy + (long long)m * a.ld_dy + c, left);
    }
    const float rstd = a.rstd[m];
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = (i * 64 * WR + l) * kPiece;
      Piece<W> pw;
      pw.load(weight + c, a.H - c);
      float n[kPiece], g[kPiece], wt[kPiece];
      pr[i].values(n);
      pg[i].values(g);
      pw.values(wt);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        n[j] *= rstd;
        dw[i][j] = __builtin_fmaf(g[j], n[j], dw[i][j]);
        dot = __builtin_fmaf(g[j] * wt[j], n[j], dot);
      }
    }
    const float mean = norm_sum<WR>(dot, reinterpret_cast<float*>(lds)) / (float)a.H;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = (i * 64 * WR + l) * kPiece, left = a.H - c;
      Piece<W> pw;
      pw.load(weight + c, left);
      float n[kPiece], g[kPiece], wt[kPiece];
      pr[i].values(n);
      pg[i].values(g);
      pw.values(wt);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) g[j] = rstd * (g[j] * wt[j] - n[j] * rstd * mean);
      if (dsum) {
        Piece<T> ps;
        ps.load(dsum + (long long)m * a.ld_dsum + c, left);
        ps.values(wt);
#pragma unroll
        for (int j = 0; j < kPiece; ++j) g[j] += wt[j];
      }
      Piece<T> o;
      o.set(g);
      o.store(dx + (long long)m * a.ld_dx + c, left);
    }
  }
  if constexpr (WR == 1) {   // the wavefronts' sums in a fixed order
    if (w > 0)
#pragma unroll
      for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < kPiece; ++j) join[w - 1][(i * kPiece + j) * 64 + lane] = dw[i][j];
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < kPiece; ++j)
#pragma unroll
        for (int o = 0; o < 3; ++o) dw[i][j] += join[o][(i * kPiece + j) * 64 + lane];
  }
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = (i * 64 * WR + l) * kPiece;
    Piece<float> o;
    o.set(dw[i]);
    o.store(a.part + (long long)blockIdx.x * a.H + c, a.H - c);
  }
}

// dweight: the workgroups' sums added in FP64 in a fixed order, 32 columns a
// workgroup, 32 of the sums' rows at a time.
constexpr int kNormSumThreads = 1024;
__global__ __launch_bounds__(kNormSumThreads) void rms_norm_weight_kernel(const float* __restrict__ part,
                                                                          float* __restrict__ dweight, int rows, int H) {
  __shared__ double lds[32][33];
  const int c = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int col = (int)blockIdx.x * 32 + c;
  double s = 0.0;
  if (col < H)
    for (int i = g; i < rows; i += 32) s += (double)part[(long long)i * H + col];
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
