// Products of E4M3 operands with an FP32 scale for each block of 128 (the
// definition is at moe_decode_matmul_fp8 in include/moe_decode.h), for one
// matrix and for the experts' matrices on rows sorted by expert.
//
// The matrix-core instruction is v_mfma_f32_16x16x128_f8f6f4: its K of 128 is
// one scale block, so one instruction forms a 16 x 16 tile's unscaled sum of a
// block from zero, and four v_fma_f32 per lane scale it into the FP32
// accumulators.  Inside that instruction (as in every FP8 one of this chip)
// eight neighbouring products are added together first, aligned to the
// largest of them and cut off 2^-13 below it (probed on the device): on
// normally distributed codes a block's sum is off by 1.5e-5 of its root mean
// square, 1/130 of the half step of a bf16 result and 1/16 of an FP16 one's,
// and never by more than 7/8 * 2^-10 of the sum of the products' magnitudes.
// An FP32 result would show it: there the codes are converted to bf16, which
// is exact, and multiplied by v_mfma_f32_16x16x32_bf16, whose sums are FP32
// (1e-8 on the same data), at half the rate.
// W is the first operand and X the second: lane l then holds
// row m = l % 16 of y and four neighbouring columns n = 4 (l / 16) + i, so a
// tile needs one scale per lane (sx[m] sw, sw being the same for the tile's
// whole 128-column block), and the four results are neighbours in y.
//
// Both operands' lanes hold 32 bytes of a row's 128: pieces (16 bytes) q and
// q + 4 for lane quarter q = l / 16.  The order of K inside a block does not
// matter as long as both operands use the same one.
#pragma once

#include "prims.hpp"

namespace moe {

constexpr int kMmBlock = 128;          // elements of K, and columns of w, that share a scale
constexpr int kMmMaxExperts = 1024;
constexpr int kMmMaxExpertRows = 1 << 24;

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 half_t;

struct MatmulArgs {
  const uint8_t* x;
  long long ldx;
  const float* sx;
  const int32_t* x_rows;   // nullptr: row m of y comes from row m of x
  const int32_t* counts;   // nullptr: one matrix
  const uint8_t* w;
  const float* sw;
  void* y;
  long long ldy;
  int X, M, N, K, E, kb, nb;   // kb, nb: blocks along K and N
  bool wide;                   // y's rows take 4-element stores
};

// The rows of y that m-tile t of BM rows covers, and their expert.
struct RowTile {
  int expert, first, rows;   // rows == 0: there is no such tile
};

// With experts, every expert's rows are cut into tiles of their own.  One
// wavefront looks at 64 experts at a time: a prefix sum over the lanes gives
// each expert's first tile and first row.
template <int BM>
__device__ __forceinline__ RowTile find_rows(const MatmulArgs& a, int t, int lane) {
  if (!a.counts) return {0, t * BM, min(BM, a.M - t * BM)};
  int tiles0 = 0, rows0 = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    const int e = e0 + lane;
    const int c = e < a.E ? min(max(a.counts[e], 0), a.M) : 0;
    const int r1 = rows0 + wave_incl_scan(c), r0 = r1 - c;
    const int used = min(r1, a.M) - min(r0, a.M);        // rows beyond M are not computed
    const int n = (used + BM - 1) / BM;
    const int t1 = tiles0 + wave_incl_scan(n);
    const uint64_t hit = __builtin_amdgcn_ballot_w64(t < t1);
    if (hit) {
      const int at = (int)__builtin_ctzll(hit);
      const int i = t - (__builtin_amdgcn_readlane(t1, at) - __builtin_amdgcn_readlane(n, at));
      const int first = __builtin_amdgcn_readlane(r0, at) + i * BM;
      return {e0 + at, first, min(BM, __builtin_amdgcn_readlane(used, at) - i * BM)};
    }
    tiles0 = __builtin_amdgcn_readlane(t1, 63);
    rows0 = min(__builtin_amdgcn_readlane(r1, 63), a.M);
  }
  return {0, 0, 0};
}

// 8 E4M3 codes -> 8 bf16 (exact).
typedef __bf16 mm_bf16x8 __attribute__((ext_vector_type(8)));
__device__ __forceinline__ mm_bf16x8 codes_to_bf16(int lo, int hi) {
  struct { bf16x2_t v[4]; } t{{e4m3x2_to_bf16x2((uint32_t)lo, false), e4m3x2_to_bf16x2((uint32_t)lo, true),
                               e4m3x2_to_bf16x2((uint32_t)hi, false), e4m3x2_to_bf16x2((uint32_t)hi, true)}};
  return __builtin_bit_cast(mm_bf16x8, t);
}

// One block's unscaled sums of a 16 x 16 tile: exact to FP32, or to what the FP8 instruction keeps.
template <bool EXACT>
__device__ __forceinline__ f32x4 block_product(const i32x8_t& w, const i32x8_t& x) {
  f32x4 p{0, 0, 0, 0};
  if constexpr (EXACT) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_to_bf16(w[2 * i], w[2 * i + 1]),
                                                  codes_to_bf16(x[2 * i], x[2 * i + 1]), p, 0, 0, 0);
    return p;
  } else {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, p, 0, 0, 0, 0, 0, 0);
  }
}

template <typename O>
__device__ __forceinline__ void store4(O* p, const f32x4& v, int left, bool wide) {
  if (wide && left >= 4) {
    if constexpr (sizeof(O) == 4) {
      *reinterpret_cast<float4*>(p) = float4{v[0], v[1], v[2], v[3]};
    } else {
      O t[4] = {(O)v[0], (O)v[1], (O)v[2], (O)v[3]};
      *reinterpret_cast<uint2*>(p) = __builtin_bit_cast(uint2, t);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) p[i] = (O)v[i];
  }
}

// A 64 x 64 tile of y per workgroup, 4 wavefronts of 32 x 32.  The 64 rows of
// each operand are staged through registers into LDS, one block of K at a
// time; piece p of row r lies at position p ^ (r % 8), so that the 16 rows of
// one operand read fall into different banks.
constexpr int kMm64 = 64;
template <typename O>
__global__ __launch_bounds__(256) void matmul_64_kernel(MatmulArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2][kMm64 * kMmBlock];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int lr = lane & 15, lq = lane >> 4;
  const int n_tiles = (a.N + kMm64 - 1) / kMm64;
  const int mt = (int)blockIdx.x / n_tiles, nt = (int)blockIdx.x - mt * n_tiles;
  const RowTile rt = find_rows<kMm64>(a, mt, lane);
  if (rt.rows <= 0) return;
  const int n0 = nt * kMm64;
  const uint8_t* wm = a.w + (size_t)rt.expert * a.N * a.K;
  const float* sw = a.sw + ((size_t)rt.expert * a.nb + n0 / kMmBlock) * a.kb;

  // this thread's two pieces of each operand: rows tid / 8 and tid / 8 + 32, piece tid % 8
  const int piece = tid & 7;
  const uint8_t* src[2][2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = (tid >> 3) + 32 * j;
    const int m = rt.first + min(r, rt.rows - 1);
    const int xr = a.x_rows ? a.x_rows[m] : m;
    src[0][j] = a.x + (long long)((unsigned)xr < (unsigned)a.X ? xr : 0) * a.ldx + 16 * piece;
    src[1][j] = wm + (size_t)min(n0 + r, a.N - 1) * a.K + 16 * piece;
  }
  // this lane's rows of y
  const float* sx[2];
  bool bad[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = 32 * (w & 1) + 16 * j + lr;
    const int m = rt.first + min(r, rt.rows - 1);
    const int xr = a.x_rows ? a.x_rows[m] : m;
    bad[j] = (unsigned)xr >= (unsigned)a.X;
    sx[j] = a.sx + (long long)(bad[j] ? 0 : xr) * a.kb;
  }

  f32x4 acc[2][2];   // [columns][rows]
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  for (int b = 0; b < a.kb; ++b) {
    u32x4 v[2][2];
    const bool in = b * kMmBlock + 16 * piece < a.K;   // K ends at a piece's edge; zeros beyond
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        v[o][j] = u32x4{{0, 0, 0, 0}};
        if (in) v[o][j] = *reinterpret_cast<const u32x4*>(src[o][j] + (size_t)b * kMmBlock);
      }
    __syncthreads();
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = (tid >> 3) + 32 * j;
        *reinterpret_cast<u32x4*>(&lds[o][r * kMmBlock + 16 * (piece ^ (r & 7))]) = v[o][j];
      }
    __syncthreads();
    i32x8_t f[2][2];
#pragma unroll
    for (int o = 0; o < 2; ++o)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int r = 32 * (o ? w >> 1 : w & 1) + 16 * j + lr;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4 t = *reinterpret_cast<const u32x4*>(&lds[o][r * kMmBlock + 16 * ((lq + 4 * h) ^ (r & 7))]);
#pragma unroll
          for (int i = 0; i < 4; ++i) f[o][j][4 * h + i] = (int)t.v[i];
        }
      }
    const float s = sw[b];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float sj = sx[j][b] * s;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f32x4 p = block_product<sizeof(O) == 4>(f[1][i], f[0][j]);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][j][c] = __builtin_fmaf(p[c], sj, acc[i][j][c]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int r = 32 * (w & 1) + 16 * j + lr;
    if (r >= rt.rows) continue;
    O* row = static_cast<O*>(a.y) + (long long)(rt.first + r) * a.ldy;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = n0 + 32 * (w >> 1) + 16 * i + 4 * lq;
      f32x4 v = acc[i][j];
      if (bad[j]) v = f32x4{qnan(), qnan(), qnan(), qnan()};
      store4(row + n, v, a.N - n, a.wide);
    }
  }
}

}  // namespace moe
