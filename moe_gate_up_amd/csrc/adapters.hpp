// Low-rank adapters of many requests beside a shared projection (the definition is
// at moe_decode_adapters in include/moe_decode.h).
//
// A workgroup takes up to 16 rows of one adapter and a range of the columns.
// First v = A x of its rows on the matrix cores, its wavefronts sharing out K and
// their sums added in LDS; then B v, 64 columns a wavefront at a time, added to the
// base in FP32 and rounded once.  v is not rounded to 16 bits: it goes into the
// second product as two 16-bit numbers whose sum it is to 2^-16 or better of itself
// (of the row's largest where T is FP16, scaled by a power of two into its range),
// which costs a second matrix instruction where memory is what bounds.
//
// Both operands of a product are read straight into the matrix instruction's
// registers: lane i + 16 q holds row i and K elements 16 q .. 16 q + 15 of 64, as
// two instructions' operands (which K elements they stand for does not matter as
// long as both operands agree).  The columns of the second product are dealt out
// such that a lane ends with 16 neighbouring columns of one row.
#pragma once

#include "pieces.hpp"
#include "quantize.hpp"
#include "sort_slots.hpp"

namespace moe {

constexpr int kAdThreads = 256;
constexpr int kAdWaves = kAdThreads / 64;
constexpr int kAdRows = 16;      // rows of one workgroup
constexpr int kAdCols = 64;      // columns of one wavefront at a time
constexpr int kAdStep = 64;      // K of one wavefront at a time
constexpr int kAdFew = 512;      // rows up to which the workgroups find theirs without a sort
constexpr int kAdMaxRank = 256;

typedef float ad_f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 ad_bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 ad_f16x8 __attribute__((ext_vector_type(8)));

struct AdapterArgs {
  const int32_t* ids;
  const float* scaling;
  const int32_t* order;    // more than kAdFew rows: rows sorted by adapter, those without one last
  const int32_t* counts;   // [L + 1]
  long long ld_x, ld_base, ld_y;
  int M, K, N, R, L;
  int splits, cols;        // ranges of columns and their length, a multiple of 64
};

template <typename T>
__device__ __forceinline__ ad_f32x4 ad_mfma(const u32x4& a, const u32x4& b, const ad_f32x4& c) {
  if constexpr (__is_same(T, f16_t))
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(ad_f16x8, a), __builtin_bit_cast(ad_f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(ad_bf16x8, a), __builtin_bit_cast(ad_bf16x8, b), c, 0, 0, 0);
}

// 8 elements at p + k, zeros from K on (K a multiple of 8); the load is always made.
template <typename T>
__device__ __forceinline__ u32x4 ad_load(const T* p, int k, int K) {
  u32x4 t = *reinterpret_cast<const u32x4*>(p + min(k, K - 8));
#pragma unroll
  for (int i = 0; i < 4; ++i) t.v[i] = k < K ? t.v[i] : 0u;
  return t;
}

// RT: 16 rows of A each, R <= 16 RT.
template <typename T, int RT, bool SORTED>
__global__ __launch_bounds__(kAdThreads) void adapters_kernel(const T* __restrict__ x, const T* __restrict__ A,
                                                              const T* __restrict__ B, const T* base, T* y,
                                                              AdapterArgs a) {
  constexpr int RP = RT * 16 < 32 ? 32 : RT * 16;   // R as the second product's steps of 32 take it
  __shared__ __attribute__((aligned(16))) float part[kAdWaves][kAdRows][RT * 16 + 4];
  __shared__ __attribute__((aligned(16))) T hi[kAdRows][RP + 8], lo[kAdRows][RP + 8];
  __shared__ float factor[kAdRows];
  __shared__ int rows[kAdRows];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int unit = (int)blockIdx.x / a.splits, c0 = ((int)blockIdx.x - unit * a.splits) * a.cols;
  const int c1 = min(c0 + a.cols, a.N);
  int ad, n = 0;   // this workgroup's adapter (-1: none) and number of rows
  if constexpr (SORTED) {
    // adapter l has ceil(counts[l] / 16) units; lane l holds `per` consecutive ones
    const int per = (a.L + 64) / 64, l0 = lane * per;
    int units = 0, total = 0;
    for (int i = 0; i < per; ++i) {
      const int c = l0 + i <= a.L ? a.counts[l0 + i] : 0;
      units += (c + kAdRows - 1) / kAdRows;
      total += c;
    }
    const int u1 = wave_incl_scan(units), r1 = wave_incl_scan(total);
    const uint64_t hit = __builtin_amdgcn_ballot_w64(unit < u1);
    if (!hit) return;   // no more units
    const int at = (int)__builtin_ctzll(hit);
    int u = __builtin_amdgcn_readlane(u1 - units, at), r = __builtin_amdgcn_readlane(r1 - total, at);
    ad = 0;
    for (int i = 0; i < per; ++i) {
      const int l = at * per + i, c = l <= a.L ? a.counts[l] : 0, k = (c + kAdRows - 1) / kAdRows;
      if (unit < u + k) {
        ad = l < a.L ? l : -1;
        r += (unit - u) * kAdRows;
        n = min(kAdRows, c - (unit - u) * kAdRows);
        break;
      }
      u += k;
      r += c;
    }
    if (tid < kAdRows) rows[tid] = a.order[r + min(tid, n - 1)];
  } else {
    // row `unit` and the next 15 of its adapter, where an even number of 16s of them lie before it
    const int mine = a.ids[unit];
    ad = (unsigned)mine < (unsigned)a.L ? mine : -1;
    int before = 0;
    for (int j0 = 0; j0 < a.M; j0 += 64) {
      const int j = j0 + lane, id = a.ids[min(j, a.M - 1)];
      const bool same = j < a.M && ((unsigned)id < (unsigned)a.L ? id : -1) == ad;
      before += __builtin_popcountll(__builtin_amdgcn_ballot_w64(same && j < unit));
      const uint64_t on = __builtin_amdgcn_ballot_w64(same && j >= unit);
      const int at = n + __builtin_popcountll(on & ((1ull << lane) - 1));
      if (w == 0 && same && j >= unit && at < kAdRows) rows[at] = j;
      n += __builtin_popcountll(on);
    }
    if (before % kAdRows) return;
    n = min(n, kAdRows);
  }
  __syncthreads();

  if (ad < 0) {
    if (base == y) return;
    for (int m = 0; m < n; ++m) {
      const long long r = rows[m];
      for (int c = c0 + tid * kPiece; c < c1; c += kAdThreads * kPiece) {
        Piece<T> p;
        if (base) {
          p.request(base + r * a.ld_base, c, a.N);
          p.settle(c, a.N);
        } else
#pragma unroll
          for (int i = 0; i < 4 * Piece<T>::kWords; ++i) p.v[i] = 0;
        p.store(y + r * a.ld_y, c, a.N);
      }
    }
    return;
  }
  const int i16 = lane & 15, q = lane >> 4;
  const long long row = rows[min(i16, n - 1)];   // this lane's row, as an operand and as a result
  const T* Aa = A + (long long)ad * a.R * a.K;
  const T* Ba = B + (long long)ad * a.N * a.R;
  {
    ad_f32x4 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = ad_f32x4{0, 0, 0, 0};
    const T* xr = x + row * a.ld_x;
    const T* ar[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) ar[t] = Aa + (long long)min(16 * t + i16, a.R - 1) * a.K;
    for (int k0 = w * kAdStep; k0 < a.K; k0 += kAdWaves * kAdStep) {
      const int k = k0 + 16 * q;
      u32x4 fx[2], fa[RT][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        fx[h] = ad_load(xr, k + 8 * h, a.K);
#pragma unroll
        for (int t = 0; t < RT; ++t) fa[t][h] = ad_load(ar[t], k + 8 * h, a.K);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int t = 0; t < RT; ++t) acc[t] = ad_mfma<T>(fa[t][h], fx[h], acc[t]);
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) *reinterpret_cast<ad_f32x4*>(&part[w][i16][16 * t + 4 * q]) = acc[t];
  }
  __syncthreads();
  {   // 16 threads a row: the wavefronts' sums, the adapter's factor, and the two halves
    const int m = tid >> 4, l = tid & 15;
    const float s = a.scaling[ad];
    float v[RP / 16], top = 0.0f;
#pragma unroll
    for (int i = 0; i < RP / 16; ++i) {
      const int r = 16 * i + l;
      v[i] = 0.0f;
      if (i < RT && r < a.R) {
#pragma unroll
        for (int o = 0; o < kAdWaves; ++o) v[i] += part[o][m][r < RT * 16 ? r : 0];
        v[i] *= s;
      }
      top = fmaxf(top, __builtin_fabsf(v[i]));
    }
    int e = 0;
    if constexpr (__is_same(T, f16_t)) {
      top = __builtin_bit_cast(float, row_max16_u32(__builtin_bit_cast(uint32_t, top)));
      if (top > 0.0f && top < __builtin_huge_valf()) e = 14 - __builtin_amdgcn_frexp_expf(top);   // below 2^14
    }
#pragma unroll
    for (int i = 0; i < RP / 16; ++i) {
      const float f = __builtin_ldexpf(v[i], e);
      const T h = (T)f;
      const float rest = f - (float)h;
      hi[m][16 * i + l] = h;
      lo[m][16 * i + l] = (T)(rest == rest ? rest : 0.0f);   // infinities have no rest
    }
    if (l == 0) factor[m] = __builtin_ldexpf(1.0f, -e);
  }
  __syncthreads();
  constexpr int S = RP / 32;
  u32x4 vh[S], vl[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    vh[s] = *reinterpret_cast<const u32x4*>(&hi[i16][32 * s + 8 * q]);
    vl[s] = *reinterpret_cast<const u32x4*>(&lo[i16][32 * s + 8 * q]);
  }
  const float back = factor[i16];
  for (int n0 = c0 + w * kAdCols; n0 < c1; n0 += kAdWaves * kAdCols) {
    ad_f32x4 acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      acc[t] = ad_f32x4{0, 0, 0, 0};
      const int nr = min(n0 + 16 * (i16 >> 2) + 4 * t + (i16 & 3), a.N - 1);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const u32x4 f = ad_load(Ba + (long long)nr * a.R, 32 * s + 8 * q, a.R);
        acc[t] = ad_mfma<T>(f, vh[s], acc[t]);
        acc[t] = ad_mfma<T>(f, vl[s], acc[t]);
      }
    }
    // this lane: row i16, columns n0 + 16 q + 4 t + j
    if (i16 >= n) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = n0 + 16 * q + 8 * h;
      if (c >= c1) continue;
      float f[kPiece];
      Piece<T> p;
      if (base) {
        p.request(base + row * a.ld_base, c, a.N);
        p.settle(c, a.N);
        p.values(f);
      }
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        const float d = acc[2 * h + j / 4][j % 4] * back;
        f[j] = base ? f[j] + d : d;
      }
      p.set(f);
      p.store(y + row * a.ld_y, c, a.N);
    }
  }
}

}  // namespace moe
