// C ABI of the low-rank adapters (adapters.hpp): argument checks, launch shapes and
// launches.  The contract is stated in include/moe_decode.h.
#include "adapters.hpp"
#include "host.hpp"
#include "moe_decode.h"

namespace {

using moe_host::aligned;
using moe_host::any_overlap;
using moe_host::rows_bytes;
using moe_host::rows_stride_ok;

constexpr int kMaxRows = 1 << 22;       // fewer
constexpr int kMaxSide = 1 << 20;       // K and N: at most
constexpr int kMaxAdapters = moe::kSortExperts - 1;
constexpr int kTargetWorkgroups = 512;

int check(int M, int K, int N, int R, int L) {
  if (M < 0 || M >= kMaxRows || K <= 0 || K % 8 || K > kMaxSide || N <= 0 || N > kMaxSide || R <= 0 || R % 8 ||
      R > moe::kAdMaxRank || L <= 0 || L > kMaxAdapters)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

// Workspace of the sort: the rows by adapter, their numbers, and the parts'.
struct Layout {
  size_t order = 0, counts = 0, before = 0, total = 0;
  Layout(int M, int L) {
    if (M <= moe::kAdFew) return;
    auto take = [&](size_t b) { const size_t r = total; total += (b + 255) & ~(size_t)255; return r; };
    order = take((size_t)M * 4);
    counts = take((size_t)(L + 1) * 4);
    before = take(moe::sort_counts(M, L + 1) * 4);
  }
};

template <typename T, int RT>
void go(hipStream_t st, const void* x, const void* A, const void* B, const void* base, void* y, moe::AdapterArgs a) {
  const bool sorted = a.M > moe::kAdFew;
  const long long units = sorted ? a.M / moe::kAdRows + (a.L + 1 < a.M ? a.L + 1 : a.M) : a.M;
  // enough workgroups for the chip; each of them repeats the first product
  const int groups = (a.N + moe::kAdCols - 1) / moe::kAdCols;
  long long s = (kTargetWorkgroups + units - 1) / units;
  const long long most = (groups + moe::kAdWaves - 1) / moe::kAdWaves;
  s = s < 1 ? 1 : s > most ? most : s;
  a.cols = (int)((groups + s - 1) / s) * moe::kAdCols;
  a.splits = (a.N + a.cols - 1) / a.cols;
  const dim3 grid((unsigned)(units * a.splits)), block(moe::kAdThreads);
  const T *px = static_cast<const T*>(x), *pa = static_cast<const T*>(A), *pb = static_cast<const T*>(B),
          *pbase = static_cast<const T*>(base);
  if (sorted) hipLaunchKernelGGL((moe::adapters_kernel<T, RT, true>), grid, block, 0, st, px, pa, pb, pbase, static_cast<T*>(y), a);
  else hipLaunchKernelGGL((moe::adapters_kernel<T, RT, false>), grid, block, 0, st, px, pa, pb, pbase, static_cast<T*>(y), a);
}
template <typename T>
void by_rank(hipStream_t st, const void* x, const void* A, const void* B, const void* base, void* y,
             const moe::AdapterArgs& a) {
  if (a.R <= 16) go<T, 1>(st, x, A, B, base, y, a);
  else if (a.R <= 32) go<T, 2>(st, x, A, B, base, y, a);
  else if (a.R <= 64) go<T, 4>(st, x, A, B, base, y, a);
  else if (a.R <= 128) go<T, 8>(st, x, A, B, base, y, a);
  else go<T, 16>(st, x, A, B, base, y, a);
}

}  // namespace

extern "C" {

int moe_decode_adapters_workspace(int M, int K, int N, int R, int L, size_t* bytes) {
  const int rc = check(M, K, N, R, L);
  if (rc) return rc;
  if (!bytes) return MOE_ERR_NULL;
  *bytes = Layout(M, L).total;
  return MOE_OK;
}

int moe_decode_adapters(const void* x, long long ld_x, int dtype, const int32_t* row_adapters, const void* a, const void* b,
                        const float* scaling, const void* base, long long ld_base, void* y, long long ld_y,
                        void* workspace, size_t workspace_bytes, int M, int K, int N, int R, int L, void* stream) {
  const int rc = check(M, K, N, R, L);
  if (rc) return rc;
  if (dtype != MOE_BF16 && dtype != MOE_F16) return MOE_ERR_ARG;
  if (M == 0) return MOE_OK;
  if (!rows_stride_ok(M, K, ld_x) || (M > 1 && ld_x % 8) || (base && !rows_stride_ok(M, N, ld_base)) ||
      !rows_stride_ok(M, N, ld_y))
    return MOE_ERR_SHAPE;
  const Layout W(M, L);
  if (!W.total) workspace = nullptr;
  if (!x || !row_adapters || !a || !b || !scaling || !y || (W.total && !workspace)) return MOE_ERR_NULL;
  if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(base, 2) || !aligned(y, 2) ||
      !aligned(row_adapters, 4) || !aligned(scaling, 4) || !aligned(workspace, 256))
    return MOE_ERR_ALIGN;
  if (W.total && workspace_bytes < W.total) return MOE_ERR_ARG;
  const bool in_place = base == y && (M <= 1 || ld_base == ld_y);
  if (any_overlap({{y, rows_bytes(M, N, ld_y, 2)}, {workspace, W.total}},
                  {{x, rows_bytes(M, K, ld_x, 2)}, {row_adapters, (size_t)M * 4}, {a, (size_t)L * R * K * 2},
                   {b, (size_t)L * N * R * 2}, {scaling, (size_t)L * 4},
                   {in_place ? nullptr : base, rows_bytes(M, N, ld_base, 2)}}) ||
      (in_place && moe_host::overlaps(workspace, W.total, base, rows_bytes(M, N, ld_base, 2))))
    return MOE_ERR_ALIAS;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  int32_t* order = reinterpret_cast<int32_t*>(ws + W.order);
  int32_t* counts = reinterpret_cast<int32_t*>(ws + W.counts);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (W.total) {
    const moe::SortArgs s{row_adapters, nullptr, counts, order, nullptr, reinterpret_cast<int32_t*>(ws + W.before), M, L + 1,
                          1, moe::sort_part(M), 0, true};
    moe::launch_sort(st, s);
  }
  const moe::AdapterArgs args{row_adapters, scaling, W.total ? order : nullptr, W.total ? counts : nullptr, ld_x, ld_base,
                              ld_y, M, K, N, R, L, 1, N};
  if (dtype == MOE_BF16) by_rank<__bf16>(st, x, a, b, base, y, args);
  else by_rank<moe::f16_t>(st, x, a, b, base, y, args);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
