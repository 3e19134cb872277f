// C ABI of the root-mean-square norm's forward pass (rms_norm.hpp): argument
// checks, launch shapes and launches.  The contract is stated in
// include/moe_decode.h.
#include "host.hpp"
#include "norm_shape.hpp"
#include "rms_norm.hpp"

namespace {

using moe_host::aligned;
using moe_host::any_overlap;
using moe_host::rows_bytes;
using moe_host::rows_stride_ok;

size_t dtype_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
bool dtype_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }

// f<WR, P>(): wavefronts of a row and pieces of a lane.  One wavefront for the shortest rows, which have no work for
// more, four as soon as they do, sixteen where four lanes' registers do not hold the row.
template <typename F>
void by_row(int H, const F& f) {
  if (H <= 512) f.template operator()<1, 1>();
  else if (H <= 1024) f.template operator()<1, 2>();
  else if (H <= 2048) f.template operator()<4, 1>();
  else if (H <= 4096) f.template operator()<4, 2>();
  else if (H <= 8192) f.template operator()<4, 4>();
  else if (H <= 16384) f.template operator()<4, 8>();
  else f.template operator()<16, 4>();
}

template <typename T, typename W>
struct Norm {
  hipStream_t st;
  const void *x, *res, *weight;
  void *y, *sum;
  const moe::NormArgs& a;
  template <int WR, int P>
  void operator()() const {
    const int rows = moe::norm_rows(WR);
    hipLaunchKernelGGL((moe::rms_norm_kernel<T, W, WR, P>), dim3((unsigned)((a.M + rows - 1) / rows)),
                       dim3((unsigned)moe::norm_threads(WR)), 0, st, static_cast<const T*>(x), static_cast<const T*>(res),
                       static_cast<const W*>(weight), static_cast<T*>(y), static_cast<T*>(sum), a);
  }
};
template <typename T>
void launch(hipStream_t st, const void* x, const void* res, const void* weight, bool f32_weight, void* y, void* sum,
            const moe::NormArgs& a) {
  if (f32_weight) by_row(a.H, Norm<T, float>{st, x, res, weight, y, sum, a});
  else by_row(a.H, Norm<T, T>{st, x, res, weight, y, sum, a});
}

}  // namespace

extern "C" int moe_decode_rms_norm(const void* x, long long ld_x, const void* residual, long long ld_residual, int dtype,
                                   const void* weight, int weight_dtype, float eps, void* y, long long ld_y, uint8_t* q,
                                   float* scales, void* sum, long long ld_sum, float* rstd, int M, int H, int flags,
                                   void* stream) {
  const int rc = moe_host::check_norm(M, H);
  if (rc) return rc;
  if (!dtype_ok(dtype) || (weight_dtype != MOE_F32 && weight_dtype != dtype) || (flags & ~MOE_QUANT_POW2) ||
      !(eps >= 0x1p-126f && eps <= 0x1p126f))
    return MOE_ERR_ARG;
  if (M == 0) return MOE_OK;
  if (!rows_stride_ok(M, H, ld_x) || (residual && !rows_stride_ok(M, H, ld_residual)) ||
      (y && !rows_stride_ok(M, H, ld_y)) || (sum && !rows_stride_ok(M, H, ld_sum)))
    return MOE_ERR_SHAPE;
  if (!x || !weight || (!y && !q) || (q && !scales) || (scales && !q) || (sum && !residual)) return MOE_ERR_NULL;
  const size_t size = dtype_size(dtype);
  if (!aligned(x, size) || !aligned(residual, size) || !aligned(weight, dtype_size(weight_dtype)) || !aligned(y, size) ||
      !aligned(sum, size) || !aligned(scales, 4) || !aligned(rstd, 4))
    return MOE_ERR_ALIGN;
  const bool in_place = sum && sum == residual && (M <= 1 || ld_sum == ld_residual);
  const size_t nb = (H + moe::kQuantBlock - 1) / moe::kQuantBlock;
  if (any_overlap({{y, rows_bytes(M, H, ld_y, size)}, {q, (size_t)M * H}, {scales, (size_t)M * nb * 4},
                   {sum, rows_bytes(M, H, ld_sum, size)}, {rstd, (size_t)M * 4}},
                  {{x, rows_bytes(M, H, ld_x, size)},
                   {in_place ? nullptr : residual, rows_bytes(M, H, ld_residual, size)},
                   {weight, (size_t)H * dtype_size(weight_dtype)}}))
    return MOE_ERR_ALIAS;
  const moe::NormArgs a{ld_x, ld_residual, ld_y, ld_sum, rstd, q, scales, M, H, eps, (flags & MOE_QUANT_POW2) != 0};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const bool f = weight_dtype == MOE_F32;
  (void)hipGetLastError();
  if (dtype == MOE_F32) by_row(H, Norm<float, float>{st, x, residual, weight, y, sum, a});
  else if (dtype == MOE_BF16) launch<__bf16>(st, x, residual, weight, f, y, sum, a);
  else launch<moe::f16_t>(st, x, residual, weight, f, y, sum, a);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}
