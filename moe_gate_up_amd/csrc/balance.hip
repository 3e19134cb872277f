// C ABI of the router's training pass (balance.hpp): argument checks, launch
// shapes and launches.  The contract is stated in include/moe_decode.h.
#include "balance.hpp"
#include "host.hpp"
#include "moe_decode.h"

namespace {

using moe_host::aligned;
using moe_host::overlaps;

int check_balance(int T, int E, int k, int G) {
  if (T < 0 || E <= 0 || k <= 0 || k > E || G <= 0) return MOE_ERR_SHAPE;
  if (E > moe::kBalMaxExperts || k > moe::kBalMaxK || T % G) return MOE_ERR_SHAPE;
  if (T > moe::kBalMaxTokens || (long long)T * k >= (1LL << 31)) return MOE_ERR_SHAPE;
  // a launch holds fewer than 2^32 threads: G * ceil(E / 32) workgroups of 1024, G (or T / 32768 and some) of 512
  if (G > (1 << 19) || (long long)G * E >= (1LL << 26)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

// One workgroup does it all, without a workspace.
bool alone(int T, int G) { return G * moe::balance_parts(T / G, G) == 1; }

size_t dtype_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }

// A row stride the byte range below cannot overflow with.
bool stride_ok(int T, int E, long long ld) { return T <= 1 || (ld >= E && ld <= (1LL << 30)); }

size_t row_bytes(int T, int E, long long ld, int dtype) {
  return ((T > 1 ? (size_t)(T - 1) * (size_t)ld : 0) + (size_t)E) * dtype_size(dtype);
}

// Whole 4-element pieces: the row starts and E allow them.
bool whole_pieces(const void* p, int T, int E, long long ld, int dtype) {
  return E % 4 == 0 && (T <= 1 || ld % 4 == 0) && aligned(p, 4 * dtype_size(dtype));
}

// f<T, LR, V, C>() for the type and the number of experts: 16 lanes a row up
// to 256 experts, else a whole wavefront.
template <typename T, int C, typename F>
void by_experts(int E, F f) {
  if (E <= 64) f.template operator()<T, 16, 4, C>();
  else if (E <= 128) f.template operator()<T, 16, 8, C>();
  else if (E <= 256) f.template operator()<T, 16, 16, C>();
  else if (E <= 512) f.template operator()<T, 64, 8, C>();
  else f.template operator()<T, 64, 16, C>();
}
template <typename F>
void by_shape(int dtype, bool whole, int E, F f) {
  if (dtype == MOE_F32) whole ? by_experts<float, 4>(E, f) : by_experts<float, 1>(E, f);
  else whole ? by_experts<uint16_t, 4>(E, f) : by_experts<uint16_t, 1>(E, f);
}

struct Forward {
  hipStream_t st;
  const void* logits;
  long long ld;
  const int32_t* ids;
  const uint8_t* valid;
  float* psum;
  int32_t* cnt;
  float* z;
  int32_t* n;
  uint32_t* ticket;
  float* losses;
  int32_t* counts;
  int32_t* tokens;
  int S, E, k, G, parts;
  template <typename T, int LR, int V, int C>
  void operator()() const {
    const dim3 grid((unsigned)(G * parts)), block(moe::kBalThreads);
    const T* x = static_cast<const T*>(logits);
    if (parts == 1 && G == 1)
      hipLaunchKernelGGL((moe::balance_parts_kernel<T, LR, V, C, true>), grid, block, 0, st, x, ld, ids, valid, psum, cnt, z,
                         n, ticket, losses, counts, tokens, S, E, k, parts);
    else
      hipLaunchKernelGGL((moe::balance_parts_kernel<T, LR, V, C, false>), grid, block, 0, st, x, ld, ids, valid, psum, cnt,
                         z, n, ticket, losses, counts, tokens, S, E, k, parts);
  }
};

struct Backward {
  hipStream_t st;
  const void* logits;
  long long ld;
  const uint8_t* valid;
  const int32_t* counts;
  const int32_t* tokens;
  const float* grad;
  void* d;
  long long ld_d;
  int S, E, k, G, parts;
  template <typename T, int LR, int V, int C>
  void operator()() const {
    hipLaunchKernelGGL((moe::balance_backward_kernel<T, LR, V, C>), dim3((unsigned)(G * parts)), dim3(moe::kBalThreads),
                       0, st, static_cast<const T*>(logits), ld, valid, counts, tokens, grad, static_cast<T*>(d), ld_d, S,
                       E, k, G, parts);
  }
};

}  // namespace

extern "C" {

int moe_decode_balance_workspace(int T, int E, int k, int G, size_t* bytes) {
  const int rc = check_balance(T, E, k, G);
  if (rc) return rc;
  if (!bytes) return MOE_ERR_NULL;
  *bytes = T == 0 || alone(T, G) ? 0 : moe::BalanceLayout(T / G, E, G).total;
  return MOE_OK;
}

int moe_decode_balance(const void* logits, long long ld, int dtype, const int32_t* topk_ids, const uint8_t* valid,
                       float* losses, int32_t* counts, int32_t* tokens, void* workspace, size_t workspace_bytes, int T,
                       int E, int k, int G, void* stream) {
  const int rc = check_balance(T, E, k, G);
  if (rc) return rc;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!stride_ok(T, E, ld)) return MOE_ERR_SHAPE;
  const bool single = alone(T, G);
  if (single) workspace = nullptr;
  if (!logits || !topk_ids || !losses || !counts || !tokens || (!single && !workspace)) return MOE_ERR_NULL;
  if (!aligned(logits, dtype_size(dtype)) || !aligned(topk_ids, 4) || !aligned(losses, 4) || !aligned(counts, 4) ||
      !aligned(tokens, 4) || !aligned(workspace, 256))
    return MOE_ERR_ALIGN;
  const moe::BalanceLayout L(T / G, E, G);
  if (!single && workspace_bytes < L.total) return MOE_ERR_ARG;
  const void* in[] = {logits, topk_ids, valid};
  const size_t inb[] = {row_bytes(T, E, ld, dtype), (size_t)T * k * 4, valid ? (size_t)T : 0};
  const void* out[] = {losses, counts, tokens, workspace};
  const size_t outb[] = {8, (size_t)G * E * 4, ((size_t)G + 1) * 4, single ? 0 : L.total};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 3; ++i)
      if (overlaps(out[o], outb[o], in[i], inb[i])) return MOE_ERR_ALIAS;
    for (int p = 0; p < o; ++p)
      if (overlaps(out[o], outb[o], out[p], outb[p])) return MOE_ERR_ALIAS;
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* psum = reinterpret_cast<float*>(ws + L.psum);
  int32_t* cnt = reinterpret_cast<int32_t*>(ws + L.cnt);
  float* z = reinterpret_cast<float*>(ws + L.z);
  int32_t* n = reinterpret_cast<int32_t*>(ws + L.n);
  uint32_t* ticket = reinterpret_cast<uint32_t*>(ws + L.ticket);
  const int S = T / G, parts = moe::balance_parts(S, G);
  hipStream_t st = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  by_shape(dtype, whole_pieces(logits, T, E, ld, dtype), E,
           Forward{st, logits, ld, topk_ids, valid, psum, cnt, z, n, ticket, losses, counts, tokens, S, E, k, G, parts});
  if (!single) {
    double* dot = reinterpret_cast<double*>(ws + L.dot);
    double* zsum = reinterpret_cast<double*>(ws + L.zsum);
    const dim3 block(moe::kBalSumThreads);
    if (E <= 128 && parts <= 128)
      hipLaunchKernelGGL(moe::balance_sum_kernel<128>, dim3((unsigned)G), block, 0, st, psum, cnt, z, n, dot, zsum, ticket,
                         losses, counts, tokens, E, k, G, parts);
    else
      hipLaunchKernelGGL(moe::balance_sum_kernel<moe::kBalSumCols>, dim3((unsigned)(G * moe::balance_splits(E))), block, 0,
                         st, psum, cnt, z, n, dot, zsum, ticket, losses, counts, tokens, E, k, G, parts);
  }
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

int moe_decode_balance_backward(const void* logits, long long ld, int dtype, const uint8_t* valid, const int32_t* counts,
                                const int32_t* tokens, const float* grad_losses, void* dlogits, long long ld_d, int T,
                                int E, int k, int G, void* stream) {
  const int rc = check_balance(T, E, k, G);
  if (rc) return rc;
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_ARG;
  if (T == 0) return MOE_OK;
  if (!stride_ok(T, E, ld) || !stride_ok(T, E, ld_d)) return MOE_ERR_SHAPE;
  if (!logits || !counts || !tokens || !grad_losses || !dlogits) return MOE_ERR_NULL;
  if (!aligned(logits, dtype_size(dtype)) || !aligned(dlogits, dtype_size(dtype)) || !aligned(counts, 4) ||
      !aligned(tokens, 4) || !aligned(grad_losses, 4))
    return MOE_ERR_ALIGN;
  const size_t db = row_bytes(T, E, ld_d, dtype);
  const void* in[] = {logits, valid, counts, tokens, grad_losses};
  const size_t inb[] = {row_bytes(T, E, ld, dtype), valid ? (size_t)T : 0, (size_t)G * E * 4, ((size_t)G + 1) * 4, 8};
  for (int i = 0; i < 5; ++i)
    if (overlaps(dlogits, db, in[i], inb[i])) return MOE_ERR_ALIAS;
  const int S = T / G, parts = moe::balance_parts(S, G);
  (void)hipGetLastError();
  by_shape(dtype, whole_pieces(logits, T, E, ld, dtype) && whole_pieces(dlogits, T, E, ld_d, dtype), E,
           Backward{static_cast<hipStream_t>(stream), logits, ld, valid, counts, tokens, grad_losses, dlogits, ld_d, S, E,
                    k, G, parts});
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
