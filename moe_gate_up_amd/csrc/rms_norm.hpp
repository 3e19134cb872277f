// Root-mean-square norm with the residual's addition and an output in 8 bits (the
// definition is at moe_decode_rms_norm in include/moe_decode.h).
//
// A row lies in the registers of WR wavefronts, P pieces of 8 columns a lane (16
// neighbouring lanes hold a block of 128 columns), so that x and the residual are
// read once and everything that is asked for is written from there, past the caches.
// The row is kept as it was rounded for `sum`: the norm is of those values.
//
// Memory bounds it.  8192 x 4096 bf16 with residual, sum, y and codes: 53.5 us, 302
// MB (5.6 TB/s; a copy 6.3).  Four wavefronts a row: one takes 70 us, two 58, eight
// 54; with results through the caches 57, with reads past them too 58.  32 x 2048:
// 3.7 us (one wavefront a row 6.4), two memory latencies and a launch.
#pragma once

#include "pieces.hpp"
#include "quantize.hpp"
#include "router.hpp"

namespace moe {

struct NormArgs {
  long long ld_x, ld_res, ld_y, ld_sum;
  float* rstd;
  uint8_t* q;
  float* scales;
  int M, H;
  float eps;
  bool pow2;
};

// Sum over the row's wavefronts, in a fixed order; every lane gets it.
template <int WR, typename A>
__device__ __forceinline__ A norm_sum(A v, A* lds) {
  if constexpr (WR == 1) {
    if constexpr (sizeof(A) == 4) return wave_sum_f32(v);
    else {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
      return v;
    }
  } else {
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if constexpr (sizeof(A) == 4) v = wave_sum_f32(v);
    else {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    }
    __syncthreads();   // an earlier sum has been read
    if (lane == 0) lds[w] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < WR; ++i) v += lds[i];
    return v;
  }
}

constexpr int norm_rows(int WR) { return WR == 1 ? 4 : 1; }          // rows of one workgroup
constexpr int norm_threads(int WR) { return WR == 1 ? 256 : 64 * WR; }

// 1 / sqrt(mean of squares + eps).  Squares that pass FP32 are added in FP64.
template <int WR, int P, typename T>
__device__ __forceinline__ float norm_rstd(const Piece<T> (&r)[P], int H, float eps, double* lds) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    float f[kPiece];
    r[i].values(f);
#pragma unroll
    for (int j = 0; j < kPiece; ++j) s = __builtin_fmaf(f[j], f[j], s);
  }
  s = norm_sum<WR>(s, reinterpret_cast<float*>(lds));
  if (s < __builtin_huge_valf()) return 1.0f / sqrtf(s / (float)H + eps);
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    float f[kPiece];
    r[i].values(f);
#pragma unroll
    for (int j = 0; j < kPiece; ++j) d = __builtin_fma((double)f[j], (double)f[j], d);
  }
  d = norm_sum<WR>(d, lds);
  return (float)(1.0 / sqrt(d / (double)H + (double)eps));
}

template <typename T, typename W, int WR, int P>
__global__ __launch_bounds__(norm_threads(WR)) void rms_norm_kernel(const T* __restrict__ x, const T* res,
                                                                    const W* __restrict__ weight, T* __restrict__ y,
                                                                    T* sum, NormArgs a) {
  __shared__ double lds[WR == 1 ? 1 : WR];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const long long m = (long long)blockIdx.x * norm_rows(WR) + (WR == 1 ? w : 0);
  if (m >= a.M) return;
  const int l = WR == 1 ? lane : (int)threadIdx.x;
  auto column = [&](int i) { return (i * 64 * WR + l) * kPiece; };
  Piece<T> r[P], t[P];
  Piece<W> wt[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    r[i].request(x + m * a.ld_x, column(i), a.H);
    if (res) t[i].request(res + m * a.ld_res, column(i), a.H);
  }
#pragma unroll
  for (int i = 0; i < P; ++i) wt[i].request(weight, column(i), a.H);
#pragma unroll
  for (int i = 0; i < P; ++i) {
    r[i].settle(column(i), a.H);
    if (res) {
      t[i].settle(column(i), a.H, res == sum ? res + m * a.ld_res : nullptr);
      float f[kPiece], g[kPiece];
      r[i].values(f);
      t[i].values(g);
#pragma unroll
      for (int j = 0; j < kPiece; ++j) f[j] += g[j];
      r[i].set(f);
      if (sum) r[i].stream(sum + m * a.ld_sum, column(i), a.H);
    }
  }
  const float rstd = norm_rstd<WR, P>(r, a.H, a.eps, lds);
  if (a.rstd && l == 0) a.rstd[m] = rstd;
  const int nb = (a.H + kQuantBlock - 1) / kQuantBlock;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    const int c = column(i), left = a.H - c;
    float f[kPiece], g[kPiece];
    wt[i].settle(c, a.H);
    r[i].values(f);
    wt[i].values(g);
#pragma unroll
    for (int j = 0; j < kPiece; ++j) f[j] = f[j] * rstd * g[j];
    if (y) {
      Piece<T> o;
      o.set(f);
      o.stream(y + m * a.ld_y, c, a.H);
    }
    if (a.q) {
#pragma unroll
      for (int j = 0; j < kPiece; ++j) f[j] = j < left ? f[j] : 0.0f;   // an infinite rstd leaves NaN there
      uint32_t lo, hi;
      const float s = block_codes(f, a.pow2, lo, hi);
      uint8_t* out = a.q + m * a.H + c;
      if (left >= kPiece) {
        typedef uint32_t any2 __attribute__((ext_vector_type(2), aligned(1)));
        __builtin_nontemporal_store(any2{lo, hi}, reinterpret_cast<any2*>(out));
      } else {
#pragma unroll
        for (int j = 0; j < kPiece; ++j)
          if (j < left) out[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
      }
      if ((l & 15) == 0 && left > 0) a.scales[m * nb + c / kQuantBlock] = s;
    }
  }
}

}  // namespace moe
