// Rows to E4M3 codes with one FP32 scale for each block of 128 columns (the
// definition is at moe_decode_quantize_fp8 in include/moe_decode.h), with the
// SwiGLU between an expert's two products as an optional prologue.
//
// One pass: 16 lanes take one block of one row, 8 elements each, so a bf16
// block is one 16-byte load per lane, the maximum is a few operations in the
// lane and 4 DPP steps, and the 8 codes are one 8-byte store.  Both divisions
// are FP32 divisions rounded correctly, so the codes equal those of the plain
// formula bit for bit: a / 448 and v / s are products with the rounded
// reciprocal and one correction from the exact residual (two fused
// multiply-adds), where a general division is ten instructions.  8192 x 4096
// bf16: 16.4 us, 102 MB (6.2 TB/s; a copy of 50 MB each way 5.9); with SwiGLU
// 32768 x 768: 21.3 us, 127 MB (6.0 TB/s).  The codes go past the caches, which
// the reads then have to themselves (18.3 and 22.7 us without; reads past the
// caches as well: 18.7 and 20.7).  Several blocks for each lane, all requested
// first, are slower than more wavefronts (one 23.0, two 24.0, four 28.1 us,
// before the divisions were trimmed).
#pragma once

#include "prims.hpp"

namespace moe {

constexpr int kQuantThreads = 256;
constexpr int kQuantBlock = 128;
constexpr int kQuantLanes = 16;    // lanes of one block
constexpr int kQuantPer = 8;       // elements of one lane
constexpr float kE4m3Max = 448.0f;
constexpr float kQuantMinScale = 0x1p-126f;

typedef _Float16 f16_t;
typedef uint32_t code_pair __attribute__((ext_vector_type(2)));

template <typename T>
__device__ __forceinline__ float elem_f32(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (__is_same(T, f16_t)) return (float)v;
  else return __builtin_bit_cast(float, (uint32_t)v << 16);
}
// How a row's pieces of 8 lie: kQuantWhole: every block is whole and its pieces
// take 16-byte loads and 8-byte stores; kQuantPieces: the last block may be
// short, by whole pieces; kQuantElements: element by element.
constexpr int kQuantWhole = 0, kQuantPieces = 1, kQuantElements = 2;

// 8 elements as FP32 from `p`, 0 from the left-th on.
template <typename T, int FORM>
__device__ __forceinline__ void load8(const T* p, int left, float (&v)[8]) {
  if constexpr (FORM == kQuantElements) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? elem_f32(p[i]) : 0.0f;
  } else {
    u32x4 raw[sizeof(T) / 2];
    const u32x4* from = reinterpret_cast<const u32x4*>(FORM == kQuantWhole ? p : p + min(left - 8, 0));   // behind K the last piece again
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) raw[i] = from[i];
    T t[8];
    __builtin_memcpy(t, raw, sizeof(t));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = FORM == kQuantWhole || left > 0 ? elem_f32(t[i]) : 0.0f;
  }
}

// Maximum over the 16 lanes of each DPP row of non-negative floats' bits.
__device__ __forceinline__ uint32_t row_max16_u32(uint32_t v) {
  v = max(v, (uint32_t)dppi<0xB1>((int)v));
  v = max(v, (uint32_t)dppi<0x4E>((int)v));
  v = max(v, (uint32_t)dppi<0x141>((int)v));
  v = max(v, (uint32_t)dppi<0x140>((int)v));
  return v;
}

// a / b rounded correctly, from the rounded reciprocal of b.
__device__ __forceinline__ float divide_by(float a, float b, float reciprocal) {
  const float t = a * reciprocal;
  return __builtin_fmaf(__builtin_fmaf(-t, b, a), reciprocal, t);
}

// SiLU(g) = g / (1 + e^-g) as n / (1 + a) with a = e^-|g| and n = g or g a, which
// cannot overflow (a below FP32's normal numbers counts as 0).  a: 2^t with t =
// -|g| log2 e rounded, and what the rounding left of the exponent added in first
// order; the quotient: the instruction's reciprocal (1 ulp) and one correction from
// the exact residual.  Times up that is within (3.5 + |g| / 43) 2^-23 of the exact
// value; t as it is and the reciprocal alone, (|g| + 4) 2^-23, took 24.2 us where
// this takes 26.7 (32768 x 768 in a graph), the reciprocal alone 26.4.
__device__ __forceinline__ float silu_exact(float g) {
  const float m = __builtin_fabsf(g), t = m * -1.44269502f, e = __builtin_amdgcn_exp2f(t);
  const float a = __builtin_fmaf(e, __builtin_fmaf(t, -0.693147182f, -m), e);
  const float n = g >= 0.0f ? g : g * a, d = 1.0f + a, r = __builtin_amdgcn_rcpf(d), q = n * r;
  const float v = __builtin_fmaf(__builtin_fmaf(-d, q, n), r, q);
  return g == -__builtin_huge_valf() ? -0.0f : v;
}

// Unit u = block u % nb of row u / nb; `magic` is ceil(2^32 / nb).
template <typename T, bool SWIGLU, int FORM>
__global__ __launch_bounds__(kQuantThreads) void quantize_kernel(const T* __restrict__ x, long long ldx,
                                                                 uint8_t* __restrict__ q, float* __restrict__ scales,
                                                                 int units, int K, int nb, uint32_t magic, bool pow2) {
  const int l = threadIdx.x & 15;
  const int u = (int)blockIdx.x * (kQuantThreads / kQuantLanes) + (int)(threadIdx.x / kQuantLanes);
  if (u >= units) return;
  int m = nb == 1 ? u : (int)__umulhi((uint32_t)u, magic);   // the quotient, or one more
  m -= m * nb > u ? 1 : 0;
  const int c = (u - m * nb) * kQuantBlock + l * kQuantPer, left = K - c;
  const T* row = x + (long long)m * ldx + c;
  float v[8];
  load8<T, FORM>(row, left, v);
  if constexpr (SWIGLU) {
    float up[8];
    load8<T, FORM>(row + K, left, up);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = silu_exact(v[j]) * up[j];
  }
  auto magnitude = [](float f) { return __builtin_bit_cast(uint32_t, f) & 0x7FFFFFFFu; };
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = max(a, magnitude(v[j]));
  a = row_max16_u32(a);
  const bool odd = a >= 0x7F800000u;   // a NaN or an infinity in the block: not part of the maximum
  uint32_t nan = 0;                    // which of this lane's 8
  if (odd) {
    a = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t t = magnitude(v[j]);
      a = max(a, t < 0x7F800000u ? t : 0u);
      nan |= t < 0x7F800000u ? 0u : 1u << j;
    }
    a = row_max16_u32(a);
  }
  float s = fmaxf(divide_by(__builtin_bit_cast(float, a), kE4m3Max, 1.0f / kE4m3Max), kQuantMinScale);
  if (pow2) {   // the next power of two: mantissa bits carry into the exponent
    const uint32_t t = __builtin_bit_cast(uint32_t, s);
    s = __builtin_bit_cast(float, (t + 0x007FFFFFu) & 0x7F800000u);
  }
  float d = s;
  if (s < 0x1p-90f) {   // keep the residuals below out of the subnormal range (exact: the block is tiny)
    d = s * 0x1p64f;
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= 0x1p64f;
  }
  const float inv = 1.0f / d;
  float r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = __builtin_copysignf(divide_by(v[j], d, inv), v[j]);   // -0 stays -0
  uint32_t lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], 0, false);
  lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], (int)lo, true);
  uint32_t hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[4], r[5], 0, false);
  hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[6], r[7], (int)hi, true);
  if (odd) {   // NaN and infinities are the one NaN code 0x7F
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t mask = 0xFFu << (8 * (j & 3)), code = 0x7Fu << (8 * (j & 3));
      if (j < 4) lo = (nan >> j & 1) ? (lo & ~mask) | code : lo;
      else hi = (nan >> j & 1) ? (hi & ~mask) | code : hi;
    }
  }
  uint8_t* out = q + (long long)m * K + c;
  if constexpr (FORM == kQuantElements) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) out[j] = (uint8_t)((j < 4 ? lo : hi) >> (8 * (j & 3)));
  } else {
    if (FORM == kQuantWhole || left > 0)
      __builtin_nontemporal_store(code_pair{lo, hi}, reinterpret_cast<code_pair*>(out));
  }
  if (l == 0) scales[u] = s;
}

}  // namespace moe
