// Rows to E4M3 codes with one FP32 scale for each block of 128 columns (the
// definition is at moe_decode_quantize_fp8 in include/moe_decode.h), with the
// SwiGLU between an expert's two products as an optional prologue.
//
// One pass, bound by memory: 16 lanes take one block of one row, 8 elements
// each, so a bf16 block is one 16-byte load per lane, the maximum is 7
// operations in the lane and 4 DPP steps, and the 8 codes are one 8-byte
// store.  Both divisions are FP32 divisions rounded correctly, so the codes
// equal those of the plain formula bit for bit: v / s is v * (1/s) with one
// correction step from the exact residual (two fused multiply-adds), a
// quarter of the instructions of a general division.
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

// 8 elements as FP32 from `p` (whole: a piece of 8 with 16-byte loads; else
// element by element, 0 from column `left` on).
template <typename T>
__device__ __forceinline__ float elem_f32(T v) {
  if constexpr (sizeof(T) == 4) return v;
  else if constexpr (__is_same(T, f16_t)) return (float)v;
  else return __builtin_bit_cast(float, (uint32_t)v << 16);
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, int left, bool whole, float (&v)[8]) {
  if (whole) {
    u32x4 raw[sizeof(T) / 2];
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) raw[i] = u32x4{{0, 0, 0, 0}};
    if (left > 0) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) raw[i] = reinterpret_cast<const u32x4*>(p)[i];
    }
    T t[8];
    __builtin_memcpy(t, raw, sizeof(t));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = elem_f32(t[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? elem_f32(p[i]) : 0.0f;
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

template <typename T, bool SWIGLU>
__global__ __launch_bounds__(kQuantThreads) void quantize_kernel(const T* __restrict__ x, long long ldx,
                                                                 uint8_t* __restrict__ q, float* __restrict__ scales,
                                                                 int units, int K, int nb, bool pow2, bool whole) {
  const int lane = threadIdx.x & 63, l = lane & 15;
  const int stride = (int)gridDim.x * (kQuantThreads / kQuantLanes);
  for (int u = (int)blockIdx.x * (kQuantThreads / kQuantLanes) + (int)(threadIdx.x / kQuantLanes); u < units; u += stride) {
    const int m = u / nb, b = u - m * nb;
    const int c = b * kQuantBlock + l * kQuantPer;
    const int left = K - c;
    const T* row = x + (long long)m * ldx;
    float v[8];
    load8(row + c, left, whole, v);
    if constexpr (SWIGLU) {
      float up[8];
      load8(row + K + c, left, whole, up);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = silu(v[i]) * up[i];
    }
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = max(a, __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu);
    a = row_max16_u32(a);
    if (a >= 0x7F800000u) {   // a NaN or an infinity in the block: not part of the maximum
      a = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t t = __builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu;
        a = max(a, t < 0x7F800000u ? t : 0u);
      }
      a = row_max16_u32(a);
    }
    float s = fmaxf(__builtin_bit_cast(float, a) / kE4m3Max, kQuantMinScale);
    if (pow2) {   // the next power of two: mantissa bits carry into the exponent
      const uint32_t t = __builtin_bit_cast(uint32_t, s);
      s = __builtin_bit_cast(float, (t + 0x007FFFFFu) & 0x7F800000u);
    }
    float d = s;
    if (s < 0x1p-90f) {   // keep the residuals below out of the subnormal range (exact: the block is tiny)
      d = s * 0x1p64f;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= 0x1p64f;
    }
    const float inv = 1.0f / d;
    float r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = v[i] * inv;
      r[i] = __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-t, d, v[i]), inv, t), v[i]);   // -0 stays -0
    }
    uint32_t lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[0], r[1], 0, false);
    lo = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[2], r[3], (int)lo, true);
    uint32_t hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[4], r[5], 0, false);
    hi = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(r[6], r[7], (int)hi, true);
    // NaN and infinities are the one NaN code 0x7F
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool bad = (__builtin_bit_cast(uint32_t, v[i]) & 0x7FFFFFFFu) >= 0x7F800000u;
      const uint32_t mask = 0xFFu << (8 * (i & 3)), nan = 0x7Fu << (8 * (i & 3));
      if (i < 4) lo = bad ? (lo & ~mask) | nan : lo;
      else hi = bad ? (hi & ~mask) | nan : hi;
    }
    uint8_t* out = q + (long long)m * K + c;
    if (whole) {
      if (left > 0) *reinterpret_cast<uint2*>(out) = uint2{lo, hi};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) out[i] = (uint8_t)((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
    if (l == 0) scales[(long long)m * nb + b] = s;
  }
}

}  // namespace moe
