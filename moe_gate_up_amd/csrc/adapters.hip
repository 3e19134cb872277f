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

int rank_tiles(int R) { return R <= 16 ? 1 : R <= 32 ? 2 : R <= 64 ? 4 : R <= 128 ? 8 : 16; }
// One launch, or three: a workgroup of the one reads all of A of its adapter, and each row of the batch is a workgroup
// (or sixteen are).  In a graph, us, mixed adapters, one launch against three: R = 16, K = 2048 (N = 4096) 1 row 7.0, 32
// 7.4 / 12.5, 384 16.1 / 17.4, 512 18.2 / 17.8 and with 16 rows for each adapter 30 / 17; R = 32, K = 1024 384 10.2 / 13.0; R =
// 64, K = 4096 1 row 22.7 / 14.6, 128 32 / 15.7; R = 128, K = 4096 36 / 18.  The rule does not know the rows' adapters, which
// the host does not see: with one for all rows (R = 16, K = 2048) 128 rows 12, 256 18, 320 and 384 30, and 385, three launches, 20.
bool few(int M, int K, int R) {
  const long long a = 16LL * rank_tiles(R) * K;
  return M <= moe::kAdFew && a <= 1 << 17 && M * a <= 3 << 22;
}
// At most: full units, and one that is not for each adapter and for none.
long long units_of(int M, int L, int rows) { return M / rows + (L + 1 < M ? L + 1 : M); }
// Shares of K: enough workgroups for the chip, each of what it takes at a time at least.
int shares_of(int M, int K, int R, int L) {
  const long long units = units_of(M, L, moe::kAdInner), want = (kTargetWorkgroups / 2 + units - 1) / units;
  const int most = (K + moe::ad_span(rank_tiles(R)) - 1) / moe::ad_span(rank_tiles(R));
  return (int)(want < most ? want : most);
}
// Rows of v that no call of up to M rows passes, so that one workspace does for all smaller batches: M times the shares is
// M (1 + floor(255 / units)) at most, where units are M or more up to L + 1 rows, and more than M / 128 + L beyond.
size_t inner_rows(int M, int K, int R, int L) {
  constexpr long long want = kTargetWorkgroups / 2 - 1;
  const long long most = (K + moe::ad_span(rank_tiles(R)) - 1) / moe::ad_span(rank_tiles(R));
  const long long of_units = want * moe::kAdInner * M / (M + (long long)moe::kAdInner * L);
  const long long rows = M + (of_units > want ? of_units : want);
  return (size_t)(rows < most * M ? rows : most * M);
}

// Workspace of many rows: their order by adapter, the adapters' numbers of rows, the sort's parts' and v.
struct Layout {
  size_t order = 0, counts = 0, before = 0, v = 0, total = 0;
  Layout(int M, int K, int R, int L) {
    if (M == 0 || few(M, K, R)) return;
    auto take = [&](size_t b) { const size_t r = total; total += (b + 255) & ~(size_t)255; return r; };
    order = take((size_t)M * 4);
    counts = take((size_t)(L + 1) * 4);
    before = take(moe::sort_counts(M, L + 1) * 4);
    v = take(inner_rows(M, K, R, L) * rank_tiles(R) * 64);
  }
};

template <typename T, int RT>
void go(hipStream_t st, const void* x, const void* A, const void* B, const void* base, void* y, moe::AdapterArgs a) {
  const T *px = static_cast<const T*>(x), *pa = static_cast<const T*>(A), *pb = static_cast<const T*>(B),
          *pbase = static_cast<const T*>(base);
  T* py = static_cast<T*>(y);
  const bool one = few(a.M, a.K, a.R);
  const long long units = one ? a.M : units_of(a.M, a.L, moe::kAdOuter);
  const int waves = one ? moe::ad_waves(RT) : moe::kAdOuterThreads / 64;
  const int target = one ? kTargetWorkgroups / 2 : 2 * kTargetWorkgroups;
  // ranges of columns: enough workgroups for the chip, of work for all their wavefronts
  const int groups = (a.N + moe::kAdCols - 1) / moe::kAdCols;
  long long s = (target + units - 1) / units;
  const long long most = (groups + waves - 1) / waves;
  s = s > most ? most : s;
  a.cols = (int)((groups + s - 1) / s) * moe::kAdCols;
  a.splits = (a.N + a.cols - 1) / a.cols;
  if (one) {
    hipLaunchKernelGGL((moe::adapters_few_kernel<T, RT>), dim3((unsigned)(units * a.splits)), dim3(64 * moe::ad_waves(RT)), 0, st,
                       px, pa, pb, pbase, py, a);
    return;
  }
  a.shares = shares_of(a.M, a.K, a.R, a.L);
  a.span = ((a.K + a.shares - 1) / a.shares + moe::kAdStep - 1) / moe::kAdStep * moe::kAdStep;
  hipLaunchKernelGGL((moe::adapters_inner_kernel<T, RT>), dim3((unsigned)(units_of(a.M, a.L, moe::kAdInner) * a.shares)),
                     dim3(4 * moe::kAdInner), 0, st, px, pa, a);
  hipLaunchKernelGGL((moe::adapters_outer_kernel<T, RT>), dim3((unsigned)(units * a.splits)), dim3(moe::kAdOuterThreads), 0, st, pb,
                     pbase, py, a);
}
template <typename T>
void by_rank(hipStream_t st, const void* x, const void* A, const void* B, const void* base, void* y,
             const moe::AdapterArgs& a) {
  switch (rank_tiles(a.R)) {
    case 1: return go<T, 1>(st, x, A, B, base, y, a);
    case 2: return go<T, 2>(st, x, A, B, base, y, a);
    case 4: return go<T, 4>(st, x, A, B, base, y, a);
    case 8: return go<T, 8>(st, x, A, B, base, y, a);
    default: return go<T, 16>(st, x, A, B, base, y, a);
  }
}

}  // namespace

extern "C" {

int moe_decode_adapters_workspace(int M, int K, int N, int R, int L, size_t* bytes) {
  const int rc = check(M, K, N, R, L);
  if (rc) return rc;
  if (!bytes) return MOE_ERR_NULL;
  *bytes = Layout(M, K, R, L).total;
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
  const Layout W(M, K, R, L);
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
  const moe::AdapterArgs args{row_adapters, scaling, order, counts, reinterpret_cast<float*>(ws + W.v), ld_x, ld_base, ld_y,
                              M, K, N, R, L, 1, N, 1, K};
  if (dtype == MOE_BF16) by_rank<__bf16>(st, x, a, b, base, y, args);
  else by_rank<moe::f16_t>(st, x, a, b, base, y, args);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
