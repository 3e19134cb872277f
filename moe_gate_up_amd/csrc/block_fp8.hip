// C ABI of the block-scaled 8-bit operators (quantize.hpp, matmul_fp8.hpp):
// argument checks, launch shapes and launches.  The contract is stated in
// include/moe_decode.h.
#include "host.hpp"
#include "matmul_fp8.hpp"
#include "moe_decode.h"
#include "quantize.hpp"

namespace {

using moe_host::aligned;
using moe_host::overlaps;

constexpr long long kMaxStride = 1LL << 30;
constexpr int kMaxSide = 1 << 30;                   // M and K: indices a tile past them are 32-bit too

// A launch holds fewer than 2^32 threads: workgroups of 256 (tiles up to 128 x 128) or up to 512.
constexpr long long max_workgroups(int variant) {
  return variant == MOE_MATMUL_ROWS_16 || variant == MOE_MATMUL_TILE_256X256 ? 1LL << 22 : 1LL << 24;
}

size_t dtype_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
bool dtype_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }
size_t row_bytes(int M, int n, long long ld, size_t size) {
  return M ? ((M > 1 ? (size_t)(M - 1) * (size_t)ld : 0) + (size_t)n) * size : 0;
}
bool stride_ok(int M, int n, long long ld) { return M <= 1 || (ld >= n && ld <= kMaxStride); }

template <typename T, bool SWIGLU, int FORM>
void go_quantize(hipStream_t st, const void* x, long long ldx, uint8_t* q, float* s, int units, int K, int nb, bool pow2) {
  constexpr int per = moe::kQuantThreads / moe::kQuantLanes;
  const uint32_t magic = (uint32_t)(((1ULL << 32) + (unsigned)nb - 1) / (unsigned)nb);   // nb = 1: not used
  hipLaunchKernelGGL((moe::quantize_kernel<T, SWIGLU, FORM>), dim3((unsigned)((units + per - 1) / per)),
                     dim3(moe::kQuantThreads), 0, st, static_cast<const T*>(x), ldx, q, s, units, K, nb, magic, pow2);
}
template <typename T, bool SWIGLU>
void pick_quantize(int form, hipStream_t st, const void* x, long long ldx, uint8_t* q, float* s, int units, int K, int nb,
                   bool pow2) {
  if (form == moe::kQuantWhole) go_quantize<T, SWIGLU, moe::kQuantWhole>(st, x, ldx, q, s, units, K, nb, pow2);
  else if (form == moe::kQuantPieces) go_quantize<T, SWIGLU, moe::kQuantPieces>(st, x, ldx, q, s, units, K, nb, pow2);
  else go_quantize<T, SWIGLU, moe::kQuantElements>(st, x, ldx, q, s, units, K, nb, pow2);
}
template <typename T>
void launch_quantize(hipStream_t st, const void* x, long long ldx, uint8_t* q, float* s, int units, int K, int nb,
                     int flags, int form) {
  const bool pow2 = flags & MOE_QUANT_POW2;
  if (flags & MOE_QUANT_SWIGLU) pick_quantize<T, true>(form, st, x, ldx, q, s, units, K, nb, pow2);
  else pick_quantize<T, false>(form, st, x, ldx, q, s, units, K, nb, pow2);
}

// ---------------------------------------------------------------- products
// A launcher returns its number of workgroups and launches only when `go` is set; `fp8`: sums of the FP8 instruction
// for a 16-bit y.
using MatmulLaunch = long long (*)(bool go, hipStream_t st, const moe::MatmulArgs& a, int y_dtype, bool fp8);

// f<O, EXACT>() for the type of y and the sums asked for.
template <typename F>
void by_result(int y_dtype, bool fp8, F f) {
  if (y_dtype == MOE_F32) f.template operator()<float, true>();
  else if (y_dtype == MOE_BF16) fp8 ? f.template operator()<__bf16, false>() : f.template operator()<__bf16, true>();
  else fp8 ? f.template operator()<moe::half_t, false>() : f.template operator()<moe::half_t, true>();
}

// Workgroups for tiles of bm x bn: with experts, each one's last tile of rows may be short, and an XCD may have up to
// two tiles more than an eighth of them.
long long tile_blocks(const moe::MatmulArgs& a, int bm, int bn) {
  const long long n_tiles = (a.N + bn - 1) / bn;
  if (!a.E) return (a.M + bm - 1) / bm * n_tiles;
  const long long tiles = (a.M / bm + (a.E < a.M ? a.E : a.M)) * n_tiles;
  return (tiles + moe::kXcds - 1) / moe::kXcds * moe::kXcds + moe::kXcds;
}

struct GoFar {
  dim3 grid;
  hipStream_t st;
  const moe::MatmulArgs& a;
  template <typename O, bool EXACT>
  void operator()() const {
    hipLaunchKernelGGL((moe::matmul_far_kernel<O, EXACT>), grid, dim3(256), 0, st, a);
  }
};
long long launch_far(bool go, hipStream_t st, const moe::MatmulArgs& a, int y_dtype, bool fp8) {
  const long long blocks = tile_blocks(a, moe::kMmFar, moe::kMmFar);
  if (go) by_result(y_dtype, fp8, GoFar{dim3((unsigned)blocks), st, a});
  return blocks;
}

template <int BM, int BN, int WM, int WN, int S, int CP>
struct GoTile {
  dim3 grid;
  hipStream_t st;
  const moe::MatmulArgs& a;
  template <typename O, bool EXACT>
  void operator()() const {
    hipLaunchKernelGGL((moe::matmul_tile_kernel<BM, BN, WM, WN, S, CP, O, EXACT>), grid, dim3(64 * WM * WN), 0, st, a);
  }
};
template <int BM, int BN, int WM, int WN, int S, int CP = moe::kCached>
long long launch_tile(bool go, hipStream_t st, const moe::MatmulArgs& a, int y_dtype, bool fp8) {
  const long long blocks = tile_blocks(a, BM, BN);
  if (go) by_result(y_dtype, fp8, GoTile<BM, BN, WM, WN, S, CP>{dim3((unsigned)blocks), st, a});
  return blocks;
}

// 16-bit results on the FP8 instruction only: FP32 sums' conversions need more registers than the accumulators leave (34
// spilled; 8192 rows, N = K = 4096 223 us, 128 x 128 229).
long long launch_256(bool go, hipStream_t st, const moe::MatmulArgs& a, int y_dtype, bool) {
  const long long blocks = tile_blocks(a, 256, 256);
  if (!go) return blocks;
  const GoTile<256, 256, 2, 4, 2, moe::kCached> f{dim3((unsigned)blocks), st, a};
  if (y_dtype == MOE_BF16) f.operator()<__bf16, false>();
  else f.operator()<moe::half_t, false>();
  return blocks;
}

template <int WK, typename O>
void go_rows(dim3 grid, hipStream_t st, const moe::MatmulArgs& a) {
  hipLaunchKernelGGL((moe::matmul_rows_kernel<WK, O>), grid, dim3(64 * WK), 0, st, a);
}
template <int WK>
long long launch_rows(bool go, hipStream_t st, const moe::MatmulArgs& a, int y_dtype, bool) {
  const long long blocks = tile_blocks(a, 16, 16);
  if (!go) return blocks;
  const dim3 grid((unsigned)blocks);
  if (y_dtype == MOE_F32) go_rows<WK, float>(grid, st, a);
  else if (y_dtype == MOE_BF16) go_rows<WK, __bf16>(grid, st, a);
  else go_rows<WK, moe::half_t>(grid, st, a);
  return blocks;
}

// The tile kernels' 32-bit offsets reach every row of a tile of bm rows.
bool tile_allowed(const moe::MatmulArgs& a, int bm) {
  return (a.x_rows ? (long long)a.X * a.ldx : (bm - 1) * a.ldx + a.K) <= (long long)moe::kMmOutOfRange;
}

// The built-in choice, from sweeps on MI355X (us in a graph; K = 2048 unless
// stated; the variants that the rule chooses between, its choice first).
// One matrix: the smallest tiles while larger ones would leave CUs without
// work, then the largest that still fill the chip.
//   16 rows: M = 1, N = 4096 4.5, 64 x 64 9.4; M = 32, N = 4096 (512
//     workgroups) 7.8, 9.8; M = 64, N = 2048, K = 4096 (512) 14.0, 17.1; but M =
//     48, N = 4096 (768) 10.7, 10.2
//   64 x 64: N = 4096, M = 256 (256 workgroups) 10.9, 64 x 128 14.4; M = 768
//     (768) 19.5, 20.9; M = 896 (896) 24.1, 21.1
//   64 x 128: N = 4096, M = 1024 (512) 21.5, 128 x 128 21.8; M = 1536 (768) 30.6,
//     31.5; M = 2048 (1024) 41.1, 33.7.  128 x 128 is not the fastest where half of
//     its columns are empty (M = 65536, K = 4096: N = 16 77.4, 64 x 64 70.8; N = 64 78.7, 76.0)
// Experts, by the tiles there can be and the rows r of an expert on average.
// 128 of 1536 x 2048, top-8:
//   64 x 64 up to 256 tiles of 64 x 128: M = 8 (96) 10.7, 64 x 128 14.0; M = 16
//     (192) 14.3, 14.7; 8 of 4096 x 2048, M = 8 (256) 13.7, 14.3, M = 64 (288) 16.8, 16.6
//   64 x 128 with w as streaming data: r = 2 55.9, cached 62.5; r = 16 71.4,
//     80.6; r = 32 87.4, 89.8; r = 40 (w is read for a second tile) 94.7, 92.8
//   128 x 128: r = 80 122.1, 64 x 128 122.6; r = 72 119.0, 115.7; r = 256 247,
//     273; not up to 512 tiles of 64 x 128: 16 of 768 x 2048, M = 2000 (282) 22.6, 16.1
int default_variant(const moe::MatmulArgs& a) {
  auto tiles = [&](int bm, int bn) { return (long long)((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
  if (a.E) {
    const int r = a.M / a.E;
    const long long most = (long long)(a.M / 64 + (a.E < a.M ? a.E : a.M)) * ((a.N + 127) / 128);
    return most <= 256 ? MOE_MATMUL_TILE_64X64
           : r <= 32 ? MOE_MATMUL_TILE_64X128_STREAM
           : r <= 79 || most <= 512 ? MOE_MATMUL_TILE_64X128 : MOE_MATMUL_TILE_128X128;
  }
  return a.M <= 16 || tiles(16, 16) <= 512 ? MOE_MATMUL_ROWS_16
         : tiles(64, 64) <= 768 ? MOE_MATMUL_TILE_64X64
         : tiles(64, 128) <= 768 ? MOE_MATMUL_TILE_64X128 : MOE_MATMUL_TILE_128X128;
}

// The same with the FP8 instruction's sums: its tiles take half the time, so larger ones pay earlier.
//   16 rows: M = 32, N = 1536 (192 workgroups) 5.8, 64 x 64 7.0; N = 2048, K =
//     4096 (256) 8.2, 10.7; but N = 4096 (512) 8.0, 7.0
//   64 x 64: N = 4096, M = 256 (256) 8.7, 64 x 128 10.1; M = 384 (384) 12.0, 10.4
//   64 x 128: N = 4096, M = 1024 (512) 15.7, 128 x 128 17.3; N = 2048, K = 4096,
//     M = 1024 16.8, 26.6; N = 4096, M = 1536 (768) 23.4, 19.1
//   256 x 256: N = 4096, M = 3000 (192) 29.8, 128 x 128 33.7; M = 2048 (128)
//     28.0, 20.5.  Not the fastest where its last round is nearly empty (N = K =
//     4096, M = 4352, 272 tiles, 108 against 97; M = 5120, 320, 108 against 102; M
//     = 6144, 384, 109 against 112) or its columns are (M = 65536, K = 4096: N =
//     16 84 against 64 x 64 67; N = 128 88 against 128 x 128 71).
// Experts:
//   64 x 64 up to 160 tiles of 64 x 128: M = 8 (96) 8.7, 64 x 128 10.2; 16 of
//     768 x 2048, M = 500 (138) 9.3, 10.8; M = 1000 (186) 12.5, 11.3
//   64 x 128 with w as streaming data: r = 2 53.9, cached 61.0; r = 16 70.4,
//     79.0; r = 32 85.8, 88.2; r = 64 122, 104; not up to 512 tiles: 8 of 4096 x
//     2048, M = 64 (288) 14.7, 13.5
//   128 x 128: r = 80 111.5, 64 x 128 114.5; r = 64 105.3, 104.8
//   256 x 256: r = 128 130.8, 128 x 128 134.8; r = 96 123.8, 119.4; r = 256 175, 200;
//     not up to 512 of its own tiles: 16 of 768 x 2048, M = 20000 (282) 48.7, 43.1; M = 40000 (516) 67.4, 79.8
int default_variant_fp8(const moe::MatmulArgs& a) {
  auto tiles = [&](int bm, int bn) { return (long long)((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn); };
  if (a.E) {
    const int r = a.M / a.E, groups = a.E < a.M ? a.E : a.M;
    auto most = [&](int bm, int bn) { return (long long)(a.M / bm + groups) * ((a.N + bn - 1) / bn); };
    return most(64, 128) <= 160 ? MOE_MATMUL_TILE_64X64
           : r <= 32 && most(64, 128) > 512 ? MOE_MATMUL_TILE_64X128_STREAM
           : r <= 71 || most(64, 128) <= 512 ? MOE_MATMUL_TILE_64X128
           : r <= 127 || most(256, 256) <= 512 ? MOE_MATMUL_TILE_128X128 : MOE_MATMUL_TILE_256X256;
  }
  return a.M <= 16 || tiles(16, 16) <= 256 ? MOE_MATMUL_ROWS_16
         : tiles(64, 64) <= 256 ? MOE_MATMUL_TILE_64X64
         : tiles(64, 128) <= 512 ? MOE_MATMUL_TILE_64X128
         : tiles(256, 256) < 192 ? MOE_MATMUL_TILE_128X128 : MOE_MATMUL_TILE_256X256;
}

// `variant` becomes the one that is launched.
MatmulLaunch matmul_launcher(int& variant, bool fp8, const moe::MatmulArgs& a, int y_dtype) {
  if (variant == 0) {
    variant = fp8 && y_dtype != MOE_F32 ? default_variant_fp8(a) : default_variant(a);
    const int bm = variant == MOE_MATMUL_TILE_256X256 ? 256 : variant == MOE_MATMUL_TILE_128X128 ? 128 : 64;
    if (variant != MOE_MATMUL_ROWS_16 && !tile_allowed(a, bm)) variant = MOE_MATMUL_FAR_ROWS;
  }
  switch (variant) {
    // 8 wavefronts along K where each of 4 would take more than 4 turns: K = 4096, M = 1 5.9 against 6.7 us; K = 2048 4.6 against 4.4
    case MOE_MATMUL_ROWS_16: return a.kb > 16 ? launch_rows<8> : launch_rows<4>;
    case MOE_MATMUL_TILE_64X64: return tile_allowed(a, 64) ? launch_tile<64, 64, 2, 2, 3> : nullptr;
    case MOE_MATMUL_TILE_64X128: return tile_allowed(a, 64) ? launch_tile<64, 128, 2, 2, 3> : nullptr;
    case MOE_MATMUL_TILE_64X128_STREAM: return tile_allowed(a, 64) ? launch_tile<64, 128, 2, 2, 3, moe::kStream> : nullptr;
    case MOE_MATMUL_TILE_128X128: return tile_allowed(a, 128) ? launch_tile<128, 128, 2, 2, 2> : nullptr;
    case MOE_MATMUL_TILE_256X256: return tile_allowed(a, 256) && y_dtype != MOE_F32 ? launch_256 : nullptr;
    case MOE_MATMUL_FAR_ROWS: return launch_far;
  }
  return nullptr;
}

int check_matmul(int X, int M, int N, int K, int E, bool experts) {
  if (M < 0 || N <= 0 || K <= 0 || X < 0 || (experts && E <= 0)) return MOE_ERR_SHAPE;
  if (K % 16 || K > kMaxSide || M >= kMaxSide || (long long)N * K >= (1LL << 31)) return MOE_ERR_SHAPE;
  if (experts && (E > moe::kMmMaxExperts || M >= moe::kMmMaxExpertRows)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

int matmul_impl(const uint8_t* x, long long ldx, const float* sx, const int32_t* x_rows, const int32_t* counts,
                const uint8_t* w, const float* sw, void* y, long long ldy, int y_dtype, int X, int M, int N, int K, int E,
                bool experts, int variant, void* stream) {
  const int rc = check_matmul(X, M, N, K, E, experts);
  if (rc) return rc;
  if (!dtype_ok(y_dtype) || variant < 0) return MOE_ERR_ARG;
  if (M == 0) return MOE_OK;
  if (X == 0 || (!x_rows && X < M) || !stride_ok(X, K, ldx) || !stride_ok(M, N, ldy)) return MOE_ERR_SHAPE;
  if (X == 1) ldx = K;   // never used
  if (M == 1) ldy = N;
  if (ldx % 16) return MOE_ERR_SHAPE;
  if (!x || !sx || !w || !sw || !y || (experts && !counts)) return MOE_ERR_NULL;
  const size_t os = dtype_size(y_dtype);
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(sx, 4) || !aligned(sw, 4) || !aligned(y, os) ||
      !aligned(x_rows, 4) || !aligned(counts, 4))
    return MOE_ERR_ALIGN;
  moe::MatmulArgs a{x, ldx, sx, x_rows, counts, w, sw, y, ldy, X, M, N, K, experts ? E : 0, (K + 127) / 128,
                    (N + 127) / 128};
  const size_t mats = experts ? (size_t)E : 1;
  const void* in[] = {x, sx, x_rows, counts, w, sw};
  const size_t inb[] = {row_bytes(X, K, ldx, 1), (size_t)X * a.kb * 4, x_rows ? (size_t)M * 4 : 0,
                        experts ? (size_t)E * 4 : 0, mats * N * K, mats * a.nb * a.kb * 4};
  for (int i = 0; i < 6; ++i)
    if (overlaps(y, row_bytes(M, N, ldy, os), in[i], inb[i])) return MOE_ERR_ALIAS;
  const bool fp8 = variant & MOE_MATMUL_FP8_SUMS;
  variant &= ~MOE_MATMUL_FP8_SUMS;
  MatmulLaunch fn = matmul_launcher(variant, fp8, a, y_dtype);
  if (!fn) return MOE_ERR_ARG;
  if (fn(false, nullptr, a, y_dtype, fp8) >= max_workgroups(variant)) return MOE_ERR_SHAPE;
  (void)hipGetLastError();
  fn(true, static_cast<hipStream_t>(stream), a, y_dtype, fp8);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // namespace

extern "C" {

int moe_decode_quantize_fp8(const void* x, long long ldx, int dtype, uint8_t* q, float* scales, int M, int K, int flags,
                            void* stream) {
  if (M < 0 || K <= 0) return MOE_ERR_SHAPE;
  if (!dtype_ok(dtype) || (flags & ~(MOE_QUANT_SWIGLU | MOE_QUANT_POW2))) return MOE_ERR_ARG;
  const bool swiglu = flags & MOE_QUANT_SWIGLU;
  if (K > (1 << 28)) return MOE_ERR_SHAPE;
  const int nb = (K + moe::kQuantBlock - 1) / moe::kQuantBlock, cols = swiglu ? 2 * K : K;
  // 16 threads each, in workgroups of 256 and a launch of fewer than 2^32
  if ((long long)M * nb > (1LL << 28) - moe::kQuantThreads / moe::kQuantLanes) return MOE_ERR_SHAPE;
  if (M == 0) return MOE_OK;
  if (!stride_ok(M, cols, ldx)) return MOE_ERR_SHAPE;
  if (!x || !q || !scales) return MOE_ERR_NULL;
  const size_t es = dtype_size(dtype);
  if (!aligned(x, es) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
  const size_t xb = row_bytes(M, cols, ldx, es), qb = (size_t)M * K, sb = (size_t)M * nb * 4;
  if (overlaps(q, qb, x, xb) || overlaps(scales, sb, x, xb) || overlaps(q, qb, scales, sb)) return MOE_ERR_ALIAS;
  const bool pieces = K % 8 == 0 && (M == 1 || (ldx * (long long)es) % 16 == 0) && aligned(x, 16) && aligned(q, 8);
  const int form = !pieces ? moe::kQuantElements : K % moe::kQuantBlock ? moe::kQuantPieces : moe::kQuantWhole;
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (dtype == MOE_F32) launch_quantize<float>(st, x, ldx, q, scales, M * nb, K, nb, flags, form);
  else if (dtype == MOE_BF16) launch_quantize<uint16_t>(st, x, ldx, q, scales, M * nb, K, nb, flags, form);
  else launch_quantize<moe::f16_t>(st, x, ldx, q, scales, M * nb, K, nb, flags, form);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

int moe_decode_matmul_fp8(const uint8_t* x, long long ldx, const float* sx, const uint8_t* w, const float* sw, void* y,
                          long long ldy, int y_dtype, int M, int N, int K, void* stream) {
  return matmul_impl(x, ldx, sx, nullptr, nullptr, w, sw, y, ldy, y_dtype, M, M, N, K, 0, false, 0, stream);
}

int moe_decode_matmul_fp8_ex(const uint8_t* x, long long ldx, const float* sx, const uint8_t* w, const float* sw, void* y,
                             long long ldy, int y_dtype, int M, int N, int K, int variant, void* stream) {
  return matmul_impl(x, ldx, sx, nullptr, nullptr, w, sw, y, ldy, y_dtype, M, M, N, K, 0, false, variant, stream);
}

int moe_decode_matmul_fp8_experts(const uint8_t* x, long long ldx, const float* sx, const int32_t* x_rows,
                                  const int32_t* counts, const uint8_t* w, const float* sw, void* y, long long ldy,
                                  int y_dtype, int X, int M, int N, int K, int E, void* stream) {
  return matmul_impl(x, ldx, sx, x_rows, counts, w, sw, y, ldy, y_dtype, X, M, N, K, E, true, 0, stream);
}

int moe_decode_matmul_fp8_experts_ex(const uint8_t* x, long long ldx, const float* sx, const int32_t* x_rows,
                                     const int32_t* counts, const uint8_t* w, const float* sw, void* y, long long ldy,
                                     int y_dtype, int X, int M, int N, int K, int E, int variant, void* stream) {
  return matmul_impl(x, ldx, sx, x_rows, counts, w, sw, y, ldy, y_dtype, X, M, N, K, E, true, variant, stream);
}

int moe_decode_matmul_fp8_plan(int M, int N, int K, int E, int* variant, int* workgroups) {
  const int rc = check_matmul(M, M, N, K, E, E != 0);
  if (rc) return rc;
  if (!variant || !workgroups) return MOE_ERR_NULL;
  moe::MatmulArgs a{};
  a.X = M, a.M = M, a.N = N, a.K = K, a.E = E, a.kb = (K + 127) / 128, a.nb = (N + 127) / 128;
  int v = 0;
  MatmulLaunch fn = matmul_launcher(v, false, a, MOE_BF16);
  const long long blocks = fn(false, nullptr, a, MOE_BF16, false);
  if (blocks >= max_workgroups(v)) return MOE_ERR_SHAPE;
  *variant = v;
  *workgroups = (int)blocks;
  return MOE_OK;
}

}  // extern "C"
