// Low-rank adapters of many requests beside a shared projection (the definition is
// at moe_decode_adapters in include/moe_decode.h).
//
// Few rows: one launch.  A workgroup takes up to 16 rows of one adapter, which it finds
// for itself, and a range of the columns.  First v = A x of its rows on the matrix
// cores, its wavefronts sharing out K and their sums added in LDS; then B v, 64 columns a
// wavefront at a time, added to the base in FP32 and rounded once.  Every range of columns
// repeats v.
// Many rows: they are sorted by adapter first, and units of rows of one adapter go
// through two launches, each of which streams: one forms v of 128 rows for a share of K, A's
// share in LDS and a wavefront's 16 rows of x requested all at once behind it; the other adds the
// shares of 32 rows and goes on as above.
//
// 32 rows with adapters of their own, 2048 -> 4096, rank 16: 7.7 us, four memory latencies
// one behind the other.  8192 rows of 8 adapters, 4096 -> 4096, rank 64: 7.2 us for the
// sort, 22 and 38 for the products of 67 and 134 MB (3.0 and 3.5 TB/s): each unit waits for
// its rows' numbers, then for its operands, and a CU holds one workgroup of the first
// product and two of the second.  Both products in one launch, 16 rows a workgroup, took
// 126: neither x nor the base was requested far enough ahead.
//
// v is not rounded to 16 bits: it goes into the second product as two 16-bit numbers
// whose sum it is to 2^-16 or better of itself (of the row's largest where T is FP16,
// scaled by a power of two into its range), which costs a second matrix instruction where
// memory is what bounds.
//
// Operands are read straight into the matrix instruction's registers: lane i + 16 q
// holds row i and 8 elements of K.  Which ones does not matter as long as both operands
// agree: two instructions' operands are pieces 2 q and 2 q + 1 of a row's 128 bytes, so
// that each load touches whole lines (halves of them took a tenth longer).
#pragma once

#include "pieces.hpp"
#include "quantize.hpp"
#include "sort_slots.hpp"

namespace moe {

constexpr int kAdRows = 16;      // rows of one workgroup, where there are few
constexpr int kAdInner = 128;    // and many: of the first product,
constexpr int kAdOuter = 32;     // and of the second
constexpr int kAdOuterThreads = 256;
constexpr int kAdCols = 64;      // columns of one wavefront at a time
constexpr int kAdStep = 64;      // K of one wavefront at a time
constexpr int kAdFew = 384;      // rows up to which the workgroups may find theirs without a sort
constexpr int kAdMaxRank = 256;

typedef float ad_f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 ad_bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 ad_f16x8 __attribute__((ext_vector_type(8)));

struct AdapterArgs {
  const int32_t* ids;
  const float* scaling;
  const int32_t* order;    // three launches: rows sorted by adapter, those without one last
  const int32_t* counts;   // [L + 1]
  float* v;                // [shares of K, M, 16 RT], in that order of rows
  long long ld_x, ld_base, ld_y;
  int M, K, N, R, L;
  int splits, cols;        // ranges of columns and their length, a multiple of 64
  int shares, span;        // shares of K and their length, a multiple of 64
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

// Wavefronts of a workgroup: 16, or as many as the LDS for their sums allows.
constexpr int ad_waves(int RT) { return RT <= 4 ? 16 : RT == 8 ? 8 : 4; }

// RT: 16 rows of A each, R <= 16 RT.
template <typename T, int RT>
__global__ __launch_bounds__(64 * ad_waves(RT)) void adapters_few_kernel(const T* __restrict__ x, const T* __restrict__ A,
                                                              const T* __restrict__ B, const T* base, T* y,
                                                              AdapterArgs a) {
  constexpr int NW = ad_waves(RT), NT = 64 * NW;
  constexpr int RP = RT * 16 < 32 ? 32 : RT * 16;   // R as the second product's steps of 32 take it
  __shared__ __attribute__((aligned(16))) float part[NW][kAdRows][RT * 16 + 4];
  __shared__ __attribute__((aligned(16))) T hi[kAdRows][RP + 8], lo[kAdRows][RP + 8];
  __shared__ float factor[kAdRows];
  __shared__ int rows[kAdRows];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int unit = (int)blockIdx.x / a.splits, c0 = ((int)blockIdx.x - unit * a.splits) * a.cols;
  const int c1 = min(c0 + a.cols, a.N);
  int ad, n = 0;   // this workgroup's adapter (-1: none) and number of rows
  {
    // row `unit` and the next 15 of its adapter, where a whole number of 16s of them lie before it
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
      for (int c = c0 + tid * kPiece; c < c1; c += NT * kPiece) {
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
  // B and the base of the first columns are requested along with x and A
  constexpr int S = RP / 32;
  constexpr bool AHEAD = S <= 2;   // as far as registers go
  Piece<T> p[2];
  u32x4 fb[AHEAD ? S : 1][4];
  auto request_base = [&](int n0) {
    if (base) {
#pragma unroll
      for (int h = 0; h < 2; ++h) p[h].request(base + row * a.ld_base, n0 + 16 * q + 8 * h, a.N);
    }
  };
  auto request_b = [&](int n0, int s) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
      fb[AHEAD ? s : 0][t] =
          ad_load(Ba + (uint32_t)min(n0 + 16 * (i16 >> 2) + 4 * t + (i16 & 3), a.N - 1) * (uint32_t)a.R, 32 * s + 8 * q, a.R);
  };
  int n0 = c0 + w * kAdCols;
  if (AHEAD) {
    request_base(n0);
#pragma unroll
    for (int s = 0; s < S; ++s) request_b(n0, s);
  }
  {
    ad_f32x4 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = ad_f32x4{0, 0, 0, 0};
    const T* xr = x + row * a.ld_x;
    const T* ar[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) ar[t] = Aa + (long long)min(16 * t + i16, a.R - 1) * a.K;
    for (int k0 = w * kAdStep; k0 < a.K; k0 += NW * kAdStep) {
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
  {   // TR threads a row: the wavefronts' sums, the adapter's factor, and the two halves
    constexpr int TR = NT / kAdRows, VR = (RP + TR - 1) / TR;
    const int m = tid / TR, l = tid % TR;
    const float s = a.scaling[ad];
    float v[VR], top = 0.0f;
#pragma unroll
    for (int i = 0; i < VR; ++i) {
      const int r = TR * i + l;
      v[i] = 0.0f;
      if (r < a.R) {
#pragma unroll
        for (int o = 0; o < NW; ++o) v[i] += part[o][m][r];
        v[i] *= s;
      }
      top = fmaxf(top, __builtin_fabsf(v[i]));
    }
    int e = 0;
    if constexpr (__is_same(T, f16_t)) {
#pragma unroll
      for (int o = TR / 2; o > 0; o /= 2) top = fmaxf(top, __shfl_xor(top, o));
      if (top > 0.0f && top < __builtin_huge_valf()) e = 14 - __builtin_amdgcn_frexp_expf(top);   // below 2^14
    }
#pragma unroll
    for (int i = 0; i < VR; ++i) {
      const int r = TR * i + l;
      if (r >= RP) continue;
      const float f = __builtin_ldexpf(v[i], e);
      const T h = (T)f;
      const float rest = f - (float)h;
      hi[m][r] = h;
      lo[m][r] = (T)(rest == rest ? rest : 0.0f);   // infinities have no rest
    }
    if (l == 0) factor[m] = __builtin_ldexpf(1.0f, -e);
  }
  __syncthreads();
  u32x4 vh[S], vl[S];
#pragma unroll
  for (int s = 0; s < S; ++s) {
    vh[s] = *reinterpret_cast<const u32x4*>(&hi[i16][32 * s + 8 * q]);
    vl[s] = *reinterpret_cast<const u32x4*>(&lo[i16][32 * s + 8 * q]);
  }
  const float back = factor[i16];
  for (bool begun = true; n0 < c1; n0 += NW * kAdCols, begun = false) {
    if (!AHEAD || !begun) request_base(n0);
    ad_f32x4 acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = ad_f32x4{0, 0, 0, 0};
#pragma unroll
    for (int s = 0; s < S; ++s) {
      if (!AHEAD || !begun) request_b(n0, s);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        acc[t] = ad_mfma<T>(fb[AHEAD ? s : 0][t], vh[s], acc[t]);
        acc[t] = ad_mfma<T>(fb[AHEAD ? s : 0][t], vl[s], acc[t]);
      }
    }
    // this lane: row i16, columns n0 + 16 q + 8 h + j
    if (i16 >= n) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = n0 + 16 * q + 8 * h;
      if (c >= c1) continue;
      float f[kPiece];
      if (base) {
        p[h].settle(c, a.N, base == y ? base + row * a.ld_base : nullptr);
        p[h].values(f);
      }
#pragma unroll
      for (int j = 0; j < kPiece; ++j) {
        const float d = acc[2 * h + j / 4][j % 4] * back;
        f[j] = base ? f[j] + d : d;
      }
      p[h].set(f);
      p[h].store(y + row * a.ld_y, c, a.N);
    }
  }
}

// This workgroup's unit of the sorted rows (adapter l has ceil(counts[l] / ROWS) of them, those without one come last)
// and which of the unit's `each` workgroups it is.  Neighbouring ones, which share an adapter's matrices, go to one
// XCD; those that there are no units for do not count in that.
struct AdUnit {
  int adapter, first, rows, part;   // -1: none; position of its first row; 0: no such unit
};
template <int ROWS>
__device__ __forceinline__ AdUnit ad_unit(const AdapterArgs& a, int each, int lane) {
  const int per = (a.L + 64) / 64, l0 = lane * per;   // lane l holds `per` consecutive adapters
  int units = 0, total = 0;
  for (int i = 0; i < per; ++i) {
    const int c = l0 + i <= a.L ? a.counts[l0 + i] : 0;
    units += (c + ROWS - 1) / ROWS;
    total += c;
  }
  const int u1 = wave_incl_scan(units), r1 = wave_incl_scan(total);
  const int all = __builtin_amdgcn_readlane(u1, 63) * each;
  if ((int)blockIdx.x >= all) return {-1, 0, 0, 0};
  const int block = xcd_contiguous_block((int)blockIdx.x, all), unit = block / each, part = block - unit * each;
  const int at = (int)__builtin_ctzll(__builtin_amdgcn_ballot_w64(unit < u1));
  int u = __builtin_amdgcn_readlane(u1 - units, at), r = __builtin_amdgcn_readlane(r1 - total, at);
  for (int l = at * per;; ++l) {   // ends within the lane's: unit < u1
    const int c = a.counts[l], k = (c + ROWS - 1) / ROWS;
    if (unit < u + k) return {l < a.L ? l : -1, r + (unit - u) * ROWS, min(ROWS, c - (unit - u) * ROWS), part};
    u += k;
    r += c;
  }
}

// K that a workgroup takes at a time: A's part of it fills 128 KB of LDS at most, x's 128 registers.
constexpr int ad_span(int RT) { return RT <= 4 ? 1024 : RT == 8 ? 512 : 256; }

// v of a share of K: a wavefront 16 rows of a unit.  Piece p of row r of A lies in LDS at place p ^ (r % 16) of its row,
// so that the 16 rows of one operand read fall into different banks.
template <typename T, int RT>
__global__ __launch_bounds__(kAdInner * 4) void adapters_inner_kernel(const T* __restrict__ x, const T* __restrict__ A,
                                                                      AdapterArgs a) {
  constexpr int SPAN = ad_span(RT), STEPS = SPAN / kAdStep, PIECES = SPAN / 8, NT = kAdInner * 4;
  __shared__ u32x4 lds[16 * RT * PIECES];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const AdUnit me = ad_unit<kAdInner>(a, a.shares, lane);
  if (me.adapter < 0) return;
  const int share = me.part;
  const int i16 = lane & 15, q = lane >> 4;
  const bool on = 16 * w < me.rows;   // of the wavefront; the others help with A
  const int at = me.first + min(16 * w + i16, me.rows - 1);
  const T* xr = x + a.order[at] * a.ld_x;
  const T* Aa = A + (long long)me.adapter * a.R * a.K;
  ad_f32x4 acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = ad_f32x4{0, 0, 0, 0};
  const int k1 = min((share + 1) * a.span, a.K);
  for (int k0 = share * a.span; k0 < k1; k0 += SPAN) {
    constexpr int EACH = 16 * RT * PIECES / NT, U = 4;   // pieces of A of a thread, requested U at a time
    u32x4 f[U], fx[STEPS][2];
    auto place = [&](int i0) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int n = (i0 + i) * NT + tid, r = n / PIECES, p = n % PIECES;
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i].v[j] = k0 + 8 * p < k1 ? f[i].v[j] : 0u;
        lds[r * PIECES + (p ^ (r & 15))] = f[i];
      }
    };
    // A before x: loads are waited for in order, and A's, from L2, would be behind all of x (24.6 us, and 21.7 so)
    for (int i0 = 0; i0 < EACH; i0 += U) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int n = (i0 + i) * NT + tid, r = n / PIECES, k = k0 + 8 * (n % PIECES);
        f[i] = *reinterpret_cast<const u32x4*>(Aa + (uint32_t)min(r, a.R - 1) * (uint32_t)a.K + (uint32_t)min(k, a.K - 8));
      }
      if (i0 + U < EACH) place(i0);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (on) {
      if (k0 + SPAN <= a.K) {   // offsets that the instructions hold: a register each spills
        const T* from = xr + (uint32_t)(k0 + 16 * q);
#pragma unroll
        for (int u = 0; u < STEPS; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h) fx[u][h] = *reinterpret_cast<const u32x4*>(from + u * kAdStep + 8 * h);
      } else {
#pragma unroll
        for (int u = 0; u < STEPS; ++u)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            fx[u][h] = *reinterpret_cast<const u32x4*>(xr + (uint32_t)min(k0 + u * kAdStep + 16 * q + 8 * h, a.K - 8));
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    place(EACH - U);
    __syncthreads();
    if (on) {
#pragma unroll
      for (int u = 0; u < STEPS; ++u) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int p = (u * kAdStep + 16 * q + 8 * h) / 8;
#pragma unroll
          for (int i = 0; i < 4; ++i) fx[u][h].v[i] = k0 + 8 * p < k1 ? fx[u][h].v[i] : 0u;
#pragma unroll
          for (int t = 0; t < RT; ++t) acc[t] = ad_mfma<T>(lds[(16 * t + i16) * PIECES + (p ^ i16)], fx[u][h], acc[t]);
        }
      }
    }
    __syncthreads();
  }
  if (16 * w + i16 >= me.rows) return;
  float* v = a.v + ((long long)share * a.M + at) * (16 * RT);
#pragma unroll
  for (int t = 0; t < RT; ++t) *reinterpret_cast<ad_f32x4*>(v + 16 * t + 4 * q) = acc[t];
}

// y of a unit and a range of columns, 64 of them a wavefront at a time.  What a wavefront reads of B and what it writes
// goes through its own part of LDS, so that neighbouring lanes access neighbouring addresses: a load of B by the matrix
// instruction's layout, 16 rows for 16 lanes, takes 64 cycles for 1 KB, and 60 % of this kernel's time went there.
// Piece p of row r of B's 8 (4) pieces lies at place p ^ (r / 2 % 8) (p ^ (r / 4 % 4)), so that 16 rows' piece p lie in
// different banks.
template <typename T, int RT>
__global__ __launch_bounds__(kAdOuterThreads) void adapters_outer_kernel(const T* __restrict__ B, const T* base, T* y,
                                                                    AdapterArgs a) {
  constexpr int RP = RT * 16 < 32 ? 32 : RT * 16, S = RP / 32, MT = kAdOuter / 16;
  constexpr int P = S == 1 ? 4 : 8, PAIRS = S == 1 ? 1 : S / 2;   // pieces of B's rows at a time, and how many times
  __shared__ __attribute__((aligned(16))) T hi[kAdOuter][RP + 8], lo[kAdOuter][RP + 8];
  __shared__ float factor[kAdOuter];
  constexpr int kSumRow = kAdCols + 4, kOwn = kAdCols * P > 4 * kSumRow ? kAdCols * P : 4 * kSumRow;
  __shared__ u32x4 own[kAdOuterThreads / 64][kOwn];   // a wavefront's B or 16 rows of sums
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const AdUnit me = ad_unit<kAdOuter>(a, a.splits, lane);
  if (me.rows == 0) return;
  const int c0 = me.part * a.cols, c1 = min(c0 + a.cols, a.N);
  if (me.adapter < 0) {
    if (base == y) return;
    for (int m = w; m < me.rows; m += kAdOuterThreads / 64) {
      const long long r = a.order[me.first + m];
      for (int c = c0 + lane * kPiece; c < c1; c += 64 * kPiece) {
        Piece<T> p;
        if (base) {
          p.request(base + r * a.ld_base, c, a.N);
          p.settle(c, a.N);
        } else {
#pragma unroll
          for (int i = 0; i < 4 * Piece<T>::kWords; ++i) p.v[i] = 0;
        }
        p.store(y + r * a.ld_y, c, a.N);
      }
    }
    return;
  }
  const int i16 = lane & 15, q = lane >> 4;
  const T* Ba = B + (long long)me.adapter * a.N * a.R;
  // as a result: rows 8 i + lane / 8, columns 8 (lane % 8) from n0 on
  constexpr int LINES = kAdOuter / 8;
  const int line = lane >> 3, col = 8 * (lane & 7);
  long long row[LINES];
#pragma unroll
  for (int i = 0; i < LINES; ++i) row[i] = a.order[me.first + min(8 * i + line, me.rows - 1)];
  // elements of K that step s of the second product has in this lane
  auto inner = [&](int s) { return S == 1 ? 8 * q : 64 * (s >> 1) + 16 * q + 8 * (s & 1); };
  u32x4* mine = own[w];
  float* sums = reinterpret_cast<float*>(mine);
  Piece<T> p[LINES];
  u32x4 f[P];   // pieces of B: row (64 j + lane) / P of 64, piece lane % P
  auto request_base = [&](int n0) {
    if (base) {
#pragma unroll
      for (int i = 0; i < LINES; ++i) p[i].request(base + row[i] * a.ld_base, n0 + col, a.N);
    }
  };
  auto request_b = [&](int n0, int pair) {
#pragma unroll
    for (int j = 0; j < P; ++j)
      f[j] = ad_load(Ba + (uint32_t)min(n0 + (64 * j + lane) / P, a.N - 1) * (uint32_t)a.R, 8 * (P * pair + lane % P), a.R);
  };
  auto place = [&](int r, int piece) { return r * P + (P == 8 ? piece ^ (r >> 1 & 7) : piece ^ (r >> 2 & 3)); };
  constexpr int STRIDE = kAdOuterThreads / 64 * kAdCols;
  int n0 = c0 + w * kAdCols;
  // before v; B first: loads are waited for in order
  request_b(n0, 0);
  __builtin_amdgcn_sched_barrier(0);
  request_base(n0);
  __builtin_amdgcn_sched_barrier(0);
  {   // 8 threads a row: the shares' sums, the adapter's factor, and the two halves
    const int m = tid >> 3, l = tid & 7, at = me.first + min(m, me.rows - 1);
    const float s = a.scaling[me.adapter];
    ad_f32x4 v[S];
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      v[i] = ad_f32x4{0, 0, 0, 0};
      const int r = 32 * i + 4 * l;
      if (r < a.R) {
#pragma unroll 4
        for (int o = 0; o < a.shares; ++o)
          v[i] += *reinterpret_cast<const ad_f32x4*>(a.v + ((long long)o * a.M + at) * (16 * RT) + r);
        v[i] *= s;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) top = fmaxf(top, __builtin_fabsf(v[i][j]));
    }
    int e = 0;
    if constexpr (__is_same(T, f16_t)) {
      top = fmaxf(top, dpp<0xB1>(top));
      top = fmaxf(top, dpp<0x4E>(top));
      top = fmaxf(top, dpp<0x141>(top));
      if (top > 0.0f && top < __builtin_huge_valf()) e = 14 - __builtin_amdgcn_frexp_expf(top);   // below 2^14
    }
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float f = __builtin_ldexpf(v[i][j], e);
        const T h = (T)f;
        const float rest = f - (float)h;
        hi[m][32 * i + 4 * l + j] = h;
        lo[m][32 * i + 4 * l + j] = (T)(rest == rest ? rest : 0.0f);   // infinities have no rest
      }
    if (l == 0) factor[m] = __builtin_ldexpf(1.0f, -e);
  }
  __syncthreads();
  while (n0 < c1) {
    ad_f32x4 acc[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[t][i] = ad_f32x4{0, 0, 0, 0};
#pragma unroll
    for (int pair = 0; pair < PAIRS; ++pair) {
      asm volatile("" ::: "memory");   // the wavefront's accesses to LDS are in order
#pragma unroll
      for (int j = 0; j < P; ++j) mine[place((64 * j + lane) / P, lane % P)] = f[j];
      asm volatile("" ::: "memory");
      if (pair + 1 < PAIRS) request_b(n0, pair + 1);
      else if (n0 + STRIDE < c1) request_b(n0 + STRIDE, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 2 * pair; s < (S == 1 ? 1 : 2 * pair + 2); ++s) {
        u32x4 g[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) g[i] = mine[place(16 * i + i16, S == 1 ? q : 2 * q + (s & 1))];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          const u32x4 vh = *reinterpret_cast<const u32x4*>(&hi[16 * t + i16][inner(s)]);
          const u32x4 vl = *reinterpret_cast<const u32x4*>(&lo[16 * t + i16][inner(s)]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            acc[t][i] = ad_mfma<T>(g[i], vh, acc[t][i]);
            acc[t][i] = ad_mfma<T>(g[i], vl, acc[t][i]);
          }
        }
      }
    }
    asm volatile("" ::: "memory");
    // 16 rows at a time through the wavefront's own part of LDS, whose accesses are in order
#pragma unroll
    for (int t = 0; t < MT; ++t) {
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<ad_f32x4*>(&sums[i16 * kSumRow + 16 * i + 4 * q]) = acc[t][i];
      asm volatile("" ::: "memory");
#pragma unroll
      for (int i = 2 * t; i < 2 * t + 2; ++i) {
        const int m = 8 * i + line;
        const float back = factor[m];
        float g[kPiece];
        if (base) {
          p[i].settle(n0 + col, a.N, base == y ? base + row[i] * a.ld_base : nullptr);
          p[i].values(g);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const ad_f32x4 d = *reinterpret_cast<const ad_f32x4*>(&sums[(m - 16 * t) * kSumRow + col + 4 * h]);
#pragma unroll
          for (int j = 0; j < 4; ++j) g[4 * h + j] = base ? __builtin_fmaf(d[j], back, g[4 * h + j]) : d[j] * back;
        }
        p[i].set(g);
        if (m < me.rows && n0 + col < c1) p[i].stream(y + row[i] * a.ld_y, n0 + col, a.N);
      }
      asm volatile("" ::: "memory");
    }
    n0 += STRIDE;
    if (n0 < c1) request_base(n0);
    __builtin_amdgcn_sched_barrier(0);
  }
}

}  // namespace moe
