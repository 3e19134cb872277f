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

size_t dtype_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
bool dtype_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }
size_t row_bytes(int M, int n, long long ld, size_t size) {
  return M ? ((M > 1 ? (size_t)(M - 1) * (size_t)ld : 0) + (size_t)n) * size : 0;
}
bool stride_ok(int M, int n, long long ld) { return M <= 1 || (ld >= n && ld <= kMaxStride); }

template <typename T>
void launch_quantize(hipStream_t st, const void* x, long long ldx, uint8_t* q, float* s, int units, int K, int nb,
                     int flags, bool whole) {
  constexpr int per = moe::kQuantThreads / moe::kQuantLanes;
  const unsigned blocks = (unsigned)((units + per - 1) / per);
  const dim3 grid(blocks < 65536u ? blocks : 65536u);
  const bool pow2 = flags & MOE_QUANT_POW2;
  const T* xt = static_cast<const T*>(x);
  if (flags & MOE_QUANT_SWIGLU)
    hipLaunchKernelGGL((moe::quantize_kernel<T, true>), grid, dim3(moe::kQuantThreads), 0, st, xt, ldx, q, s, units, K, nb,
                       pow2, whole);
  else
    hipLaunchKernelGGL((moe::quantize_kernel<T, false>), grid, dim3(moe::kQuantThreads), 0, st, xt, ldx, q, s, units, K,
                       nb, pow2, whole);
}

// ---------------------------------------------------------------- products
// A launcher returns its number of workgroups and launches only when `go` is set.
using MatmulLaunch = long long (*)(bool go, hipStream_t st, const moe::MatmulArgs& a, int y_dtype);

// m-tiles of at most BM rows: with experts, each one's last tile may be short.
long long row_tiles(const moe::MatmulArgs& a, int bm) {
  if (!a.E) return (a.M + bm - 1) / bm;
  return a.M / bm + (a.E < a.M ? a.E : a.M);
}

template <typename O>
void go_64(dim3 grid, hipStream_t st, const moe::MatmulArgs& a) {
  hipLaunchKernelGGL(moe::matmul_64_kernel<O>, grid, dim3(256), 0, st, a);
}
long long launch_64(bool go, hipStream_t st, const moe::MatmulArgs& a, int y_dtype) {
  const long long blocks = row_tiles(a, moe::kMm64) * ((a.N + moe::kMm64 - 1) / moe::kMm64);
  if (!go) return blocks;
  const dim3 grid((unsigned)blocks);
  if (y_dtype == MOE_F32) go_64<float>(grid, st, a);
  else if (y_dtype == MOE_BF16) go_64<__bf16>(grid, st, a);
  else go_64<moe::half_t>(grid, st, a);
  return blocks;
}

MatmulLaunch matmul_launcher(int& variant, const moe::MatmulArgs& a) {
  if (variant == 0) variant = MOE_MATMUL_TILE_64;
  switch (variant) {
    case MOE_MATMUL_TILE_64: return launch_64;
  }
  return nullptr;
}

int check_matmul(int X, int M, int N, int K, int E, bool experts) {
  if (M < 0 || N <= 0 || K <= 0 || X < 0 || (experts && E <= 0)) return MOE_ERR_SHAPE;
  if (K % 16 || (long long)N * K >= (1LL << 31)) return MOE_ERR_SHAPE;
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
  if (ldx % 16 || (x_rows && (long long)X * ldx >= (1LL << 32))) return MOE_ERR_SHAPE;
  if (!x || !sx || !w || !sw || !y || (experts && !counts)) return MOE_ERR_NULL;
  const size_t os = dtype_size(y_dtype);
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(sx, 4) || !aligned(sw, 4) || !aligned(y, os) ||
      !aligned(x_rows, 4) || !aligned(counts, 4))
    return MOE_ERR_ALIGN;
  moe::MatmulArgs a{x, ldx, sx, x_rows, counts, w, sw, y, ldy, X, M, N, K, experts ? E : 0, (K + 127) / 128,
                    (N + 127) / 128, N % 4 == 0 && ldy % 4 == 0 && aligned(y, 4 * os)};
  const size_t mats = experts ? (size_t)E : 1;
  const void* in[] = {x, sx, x_rows, counts, w, sw};
  const size_t inb[] = {row_bytes(X, K, ldx, 1), (size_t)X * a.kb * 4, x_rows ? (size_t)M * 4 : 0,
                        experts ? (size_t)E * 4 : 0, mats * N * K, mats * a.nb * a.kb * 4};
  for (int i = 0; i < 6; ++i)
    if (overlaps(y, row_bytes(M, N, ldy, os), in[i], inb[i])) return MOE_ERR_ALIAS;
  MatmulLaunch fn = matmul_launcher(variant, a);
  if (!fn) return MOE_ERR_ARG;
  if (fn(false, nullptr, a, y_dtype) >= (1LL << 22)) return MOE_ERR_SHAPE;   // a launch holds fewer than 2^32 threads
  (void)hipGetLastError();
  fn(true, static_cast<hipStream_t>(stream), a, y_dtype);
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
  if ((long long)M * nb >= (1LL << 30)) return MOE_ERR_SHAPE;
  if (M == 0) return MOE_OK;
  if (!stride_ok(M, cols, ldx)) return MOE_ERR_SHAPE;
  if (!x || !q || !scales) return MOE_ERR_NULL;
  const size_t es = dtype_size(dtype);
  if (!aligned(x, es) || !aligned(scales, 4)) return MOE_ERR_ALIGN;
  const size_t xb = row_bytes(M, cols, ldx, es), qb = (size_t)M * K, sb = (size_t)M * nb * 4;
  if (overlaps(q, qb, x, xb) || overlaps(scales, sb, x, xb) || overlaps(q, qb, scales, sb)) return MOE_ERR_ALIAS;
  // whole pieces of 8 elements: 16-byte loads, 8-byte stores
  const bool whole = K % 8 == 0 && (M == 1 || (ldx * (long long)es) % 16 == 0) && aligned(x, 16) && aligned(q, 8);
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (dtype == MOE_F32) launch_quantize<float>(st, x, ldx, q, scales, M * nb, K, nb, flags, whole);
  else if (dtype == MOE_BF16) launch_quantize<uint16_t>(st, x, ldx, q, scales, M * nb, K, nb, flags, whole);
  else launch_quantize<moe::f16_t>(st, x, ldx, q, scales, M * nb, K, nb, flags, whole);
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
  MatmulLaunch fn = matmul_launcher(v, a);
  *variant = v;
  *workgroups = (int)fn(false, nullptr, a, MOE_BF16);
  return MOE_OK;
}

}  // extern "C"
