// C ABI of the routing to experts by scores, of the slots sorted by expert and of
// the combination of the experts' rows (route_experts.hpp, sort_slots.hpp,
// combine.hpp): argument checks, launch shapes and launches.  The contract is
// stated in include/moe_decode.h.
#include "combine.hpp"
#include "host.hpp"
#include "moe_decode.h"
#include "route_experts.hpp"
#include "sort_slots.hpp"

namespace {

using moe_host::aligned;
using moe_host::any_overlap;
using moe_host::rows_bytes;
using moe_host::rows_stride_ok;

static_assert(MOE_ROUTE_SIGMOID == moe::kScoreSigmoid && MOE_ROUTE_RENORM == moe::kScoreRenorm &&
              MOE_ROUTE_GROUP_TOP2 == moe::kScoreTop2, "flags");
constexpr int kFlags = MOE_ROUTE_SIGMOID | MOE_ROUTE_RENORM | MOE_ROUTE_GROUP_TOP2;
constexpr int kMaxTokens = 1 << 26;   // fewer: 64 threads a token and fewer than 2^32 in a launch
constexpr int kMaxSlots = 1 << 24;    // slots of a sort, rows of a product: fewer

size_t dtype_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// Whole 4-element pieces of n elements from the rows' starts.
bool quads(const void* p, int T, int n, long long ld, int dtype) {
  return n % 4 == 0 && (T <= 1 || ld % 4 == 0) && aligned(p, 4 * dtype_size(dtype));
}

int check_route(int T, int E, int k) {
  if (T < 0 || T >= kMaxTokens || E <= 0 || E > moe::kBalMaxExperts || k <= 0 || k > moe::kBalMaxK || k > E ||
      (long long)T * k >= 1LL << 31)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

constexpr int kGrid = 1024;   // workgroups of a pass over many rows: 4 a CU, as many as stay at a time

struct Choose {
  hipStream_t st;
  const void* logits;
  const moe::ScoreArgs& a;
  template <typename T, int LR, int V, int C>
  void operator()() const {
    const int rows = moe::kScoreWaves * (64 / LR), n = (a.T + rows - 1) / rows;
    const dim3 grid((unsigned)(n < kGrid ? n : kGrid)), block(moe::kScoreThreads);
    const T* x = static_cast<const T*>(logits);
    if (!a.bias) hipLaunchKernelGGL((moe::route_experts_kernel<T, LR, V, C, moe::kByLogit>), grid, block, 0, st, x, a);
    else if (a.flags & moe::kScoreSigmoid)
      hipLaunchKernelGGL((moe::route_experts_kernel<T, LR, V, C, moe::kBySigmoid>), grid, block, 0, st, x, a);
    else hipLaunchKernelGGL((moe::route_experts_kernel<T, LR, V, C, moe::kBySoftmax>), grid, block, 0, st, x, a);
  }
};
// More than 16 of a lane: in groups, which leave lanes without an expert.
template <typename T, int LR, int C, int MOST, typename F>
void by_experts_of_lane(int n, const F& f) {
  static_assert(MOST == 16 || MOST == 32, "experts of a lane");
  if (n <= 4) f.template operator()<T, LR, 4, C>();
  else if (n <= 8) f.template operator()<T, LR, 8, C>();
  else if (n <= 16) f.template operator()<T, LR, 16, C>();
  else if constexpr (MOST > 16) f.template operator()<T, LR, 32, C>();
}
template <typename T, int LR, typename F>
void by_piece(bool whole, int n, const F& f) {
  whole ? by_experts_of_lane<T, LR, 4, 32>(n, f) : by_experts_of_lane<T, LR, 1, 32>(n, f);
}

struct RouteBackward {
  hipStream_t st;
  const void* logits;
  long long ld;
  const int32_t* ids;
  const float* grad;
  void* d;
  long long ld_d;
  int T, E, k, flags;
  float scale;
  template <typename E_, int LR, int V, int C>
  void operator()() const {
    const int rows = moe::kScoreWaves * (64 / LR);
    hipLaunchKernelGGL((moe::route_experts_backward_kernel<E_, LR, V, C>), dim3((unsigned)((T + rows - 1) / rows)),
                       dim3(moe::kScoreThreads), 0, st, static_cast<const E_*>(logits), ld, ids, grad,
                       static_cast<E_*>(d), ld_d, T, E, k, flags, scale);
  }
};
// 16 lanes a row up to 256 experts and 16 slots, else a whole wavefront.
template <typename T, int C>
void backward_by_size(int E, int k, const RouteBackward& f) {
  if (k > 16 || E > 256) by_experts_of_lane<T, 64, C, 16>((E + 63) / 64, f);
  else by_experts_of_lane<T, 16, C, 16>((E + 15) / 16, f);
}

// ---------------------------------------------------------------- slots by expert
int check_sort(int T, int E, int k) {
  if (T < 0 || E <= 0 || E > moe::kSortExperts || k <= 0 || k > moe::kBalMaxK || (long long)T * k >= kMaxSlots)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}

// ---------------------------------------------------------------- combine
bool value_type(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }
int check_combine(int M, int T, int N, int k) {
  if (M < 0 || M > kMaxSlots || T < 0 || N <= 0 || N > 1 << 28 || k <= 0 || k > moe::kCombineMaxK ||
      (long long)T * k >= kMaxSlots || (long long)T * ((N + 2047) / 2048) >= kMaxSlots)
    return MOE_ERR_SHAPE;
  return MOE_OK;
}
// Threads for pieces of 8 columns, at most a workgroup's.
int piece_threads(int N) {
  const int p = (N + moe::kPiece - 1) / moe::kPiece;
  return p >= moe::kCombineThreads ? moe::kCombineThreads : (p + 63) / 64 * 64;
}
template <typename T>
void launch_combine(hipStream_t st, const void* rows, const void* add, void* y, moe::CombineArgs a) {
  const int threads = piece_threads(a.N);
  a.chunks = (a.N + threads * moe::kPiece - 1) / (threads * moe::kPiece);
  hipLaunchKernelGGL((moe::combine_kernel<T>), dim3((unsigned)(a.T * a.chunks)), dim3((unsigned)threads), 0, st,
                     static_cast<const T*>(rows), static_cast<const T*>(add), static_cast<T*>(y), a);
}
template <typename T>
void launch_combine_backward(hipStream_t st, const void* dy, const void* rows, void* drows,
                             const moe::CombineBackwardArgs& a) {
  hipLaunchKernelGGL((moe::combine_backward_kernel<T>), dim3((unsigned)a.T), dim3((unsigned)piece_threads(a.N)), 0, st,
                     static_cast<const T*>(dy), static_cast<const T*>(rows), static_cast<T*>(drows), a);
}

int launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH; }

}  // namespace

extern "C" {

int moe_decode_route_experts(const void* logits, long long ld, int dtype, const float* bias, int32_t* topk_ids,
                             float* topk_weights, int T, int E, int k, int groups, int top_groups, int flags, float scale,
                             void* stream) {
  const int rc = check_route(T, E, k);
  if (rc) return rc;
  if (groups <= 0 || groups > 64 || groups > E || E % groups || top_groups <= 0 || top_groups > groups ||
      k > top_groups * (E / groups))
    return MOE_ERR_SHAPE;
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || (flags & ~kFlags)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!rows_stride_ok(T, E, ld)) return MOE_ERR_SHAPE;
  if (!logits || !topk_ids || !topk_weights) return MOE_ERR_NULL;
  if (!aligned(logits, dtype_size(dtype)) || !aligned(bias, 4) || !aligned(topk_ids, 4) || !aligned(topk_weights, 4))
    return MOE_ERR_ALIGN;
  const size_t slots = (size_t)T * k * 4;
  if (any_overlap({{topk_ids, slots}, {topk_weights, slots}},
                  {{logits, rows_bytes(T, E, ld, dtype_size(dtype))}, {bias, (size_t)E * 4}}))
    return MOE_ERR_ALIAS;
  // 16 lanes a row where its experts, groups and slots fit them
  if (top_groups == groups) groups = top_groups = 1;   // none is left out: no groups
  const int lanes = E > 256 || k > 16 || groups > 16 ? 64 : 16, Eg = E / groups;
  int lg = 0;
  while ((2 << lg) * groups <= lanes) ++lg;
  if (Eg == 1) flags &= ~MOE_ROUTE_GROUP_TOP2;         // the largest is all there is
  const bool whole = quads(logits, T, Eg, ld, dtype);
  const int c = whole ? 4 : 1, n = (Eg + (c << lg) - 1) / (c << lg) * c;
  const moe::ScoreArgs a{bias, topk_ids, topk_weights, ld, T, E, k, groups, Eg, top_groups, lg, flags, scale};
  const Choose f{static_cast<hipStream_t>(stream), logits, a};
  (void)hipGetLastError();
  if (dtype == MOE_F32) lanes == 16 ? by_piece<float, 16>(whole, n, f) : by_piece<float, 64>(whole, n, f);
  else lanes == 16 ? by_piece<uint16_t, 16>(whole, n, f) : by_piece<uint16_t, 64>(whole, n, f);
  return launched();
}

int moe_decode_route_experts_backward(const void* logits, long long ld, int dtype, const int32_t* topk_ids,
                                      const float* grad_weights, void* dlogits, long long ld_d, int T, int E, int k,
                                      int flags, float scale, void* stream) {
  const int rc = check_route(T, E, k);
  if (rc) return rc;
  if ((dtype != MOE_F32 && dtype != MOE_BF16) || (flags & ~kFlags)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!rows_stride_ok(T, E, ld) || !rows_stride_ok(T, E, ld_d)) return MOE_ERR_SHAPE;
  if (!logits || !topk_ids || !grad_weights || !dlogits) return MOE_ERR_NULL;
  const size_t size = dtype_size(dtype), slots = (size_t)T * k * 4;
  if (!aligned(logits, size) || !aligned(dlogits, size) || !aligned(topk_ids, 4) || !aligned(grad_weights, 4))
    return MOE_ERR_ALIGN;
  if (any_overlap({{dlogits, rows_bytes(T, E, ld_d, size)}},
                  {{logits, rows_bytes(T, E, ld, size)}, {topk_ids, slots}, {grad_weights, slots}}))
    return MOE_ERR_ALIAS;
  const RouteBackward f{static_cast<hipStream_t>(stream), logits, ld, topk_ids, grad_weights, dlogits, ld_d, T, E, k,
                        flags, scale};
  const bool whole = quads(logits, T, E, ld, dtype) && quads(dlogits, T, E, ld_d, dtype);
  (void)hipGetLastError();
  if (dtype == MOE_F32) whole ? backward_by_size<float, 4>(E, k, f) : backward_by_size<float, 1>(E, k, f);
  else whole ? backward_by_size<uint16_t, 4>(E, k, f) : backward_by_size<uint16_t, 1>(E, k, f);
  return launched();
}

int moe_decode_sort_slots_workspace(int T, int E, int k, size_t* bytes) {
  const int rc = check_sort(T, E, k);
  if (rc) return rc;
  if (!bytes) return MOE_ERR_NULL;
  *bytes = T ? moe::sort_counts(T * k, E) * 4 : 0;
  return MOE_OK;
}

int moe_decode_sort_slots(const int32_t* topk_ids, const uint8_t* valid, int32_t* counts, int32_t* x_rows,
                          int32_t* positions, void* workspace, size_t workspace_bytes, int T, int E, int k, void* stream) {
  const int rc = check_sort(T, E, k);
  if (rc) return rc;
  if (T == 0) return MOE_OK;
  const int slots = T * k;
  const size_t need = moe::sort_counts(slots, E) * 4, slot_bytes = (size_t)slots * 4;
  if (!need) workspace = nullptr;
  if (!topk_ids || !counts || !x_rows || !positions || (need && !workspace)) return MOE_ERR_NULL;
  if (!aligned(topk_ids, 4) || !aligned(counts, 4) || !aligned(x_rows, 4) || !aligned(positions, 4) ||
      !aligned(workspace, 256))
    return MOE_ERR_ALIGN;
  if (need && workspace_bytes < need) return MOE_ERR_ARG;
  if (any_overlap({{counts, (size_t)E * 4}, {x_rows, slot_bytes}, {positions, slot_bytes}, {workspace, need}},
                  {{topk_ids, slot_bytes}, {valid, (size_t)T}}))
    return MOE_ERR_ALIAS;
  const uint32_t magic = (uint32_t)(((1ULL << 32) + (unsigned)k - 1) / (unsigned)k);   // k = 1: not used
  const moe::SortArgs a{topk_ids, valid, counts, x_rows, positions, static_cast<int32_t*>(workspace), slots, E, k,
                        moe::sort_part(slots), magic, false};
  (void)hipGetLastError();
  moe::launch_sort(static_cast<hipStream_t>(stream), a);
  return launched();
}

int moe_decode_combine(const void* rows, long long ld_rows, int dtype, const int32_t* positions, const float* weights,
                       const void* add, long long ld_add, void* y, long long ld_y, int M, int T, int N, int k,
                       void* stream) {
  const int rc = check_combine(M, T, N, k);
  if (rc) return rc;
  if (!value_type(dtype)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!rows_stride_ok(M, N, ld_rows) || (add && !rows_stride_ok(T, N, ld_add)) || !rows_stride_ok(T, N, ld_y))
    return MOE_ERR_SHAPE;
  if ((!rows && M) || !positions || !y) return MOE_ERR_NULL;
  const size_t size = dtype_size(dtype), slots = (size_t)T * k * 4, out = rows_bytes(T, N, ld_y, size);
  if (!aligned(rows, size) || !aligned(add, size) || !aligned(y, size) || !aligned(positions, 4) || !aligned(weights, 4))
    return MOE_ERR_ALIGN;
  const bool in_place = add == y && (T <= 1 || ld_add == ld_y);
  if (any_overlap({{y, out}}, {{rows, rows_bytes(M, N, ld_rows, size)}, {positions, slots}, {weights, slots},
                               {in_place ? nullptr : add, rows_bytes(T, N, ld_add, size)}}))
    return MOE_ERR_ALIAS;
  const moe::CombineArgs a{positions, weights, ld_rows, ld_add, ld_y, M, T, N, k, 0};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (dtype == MOE_F32) launch_combine<float>(st, rows, add, y, a);
  else if (dtype == MOE_BF16) launch_combine<__bf16>(st, rows, add, y, a);
  else launch_combine<moe::f16_t>(st, rows, add, y, a);
  return launched();
}

int moe_decode_combine_backward(const void* dy, long long ld_dy, const void* rows, long long ld_rows, int dtype,
                                const int32_t* positions, const float* weights, void* drows, long long ld_d,
                                float* dweights, int M, int T, int N, int k, void* stream) {
  const int rc = check_combine(M, T, N, k);
  if (rc) return rc;
  if (!value_type(dtype)) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!rows_stride_ok(T, N, ld_dy) || (dweights && !rows_stride_ok(M, N, ld_rows)) || !rows_stride_ok(M, N, ld_d))
    return MOE_ERR_SHAPE;
  if (!dy || !positions || (M && (!drows || (dweights && !rows)))) return MOE_ERR_NULL;
  const size_t size = dtype_size(dtype), slots = (size_t)T * k * 4;
  if (!dweights) rows = nullptr;   // not read
  if (!aligned(dy, size) || !aligned(rows, size) || !aligned(drows, size) || !aligned(positions, 4) ||
      !aligned(weights, 4) || !aligned(dweights, 4))
    return MOE_ERR_ALIGN;
  if (any_overlap({{drows, rows_bytes(M, N, ld_d, size)}, {dweights, slots}},
                  {{dy, rows_bytes(T, N, ld_dy, size)}, {rows, rows_bytes(M, N, ld_rows, size)}, {positions, slots},
                   {weights, slots}}))
    return MOE_ERR_ALIAS;
  const moe::CombineBackwardArgs a{positions, weights, dweights, ld_dy, ld_rows, ld_d, M, T, N, k};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (dtype == MOE_F32) launch_combine_backward<float>(st, dy, rows, drows, a);
  else if (dtype == MOE_BF16) launch_combine_backward<__bf16>(st, dy, rows, drows, a);
  else launch_combine_backward<moe::f16_t>(st, dy, rows, drows, a);
  return launched();
}

}  // extern "C"
