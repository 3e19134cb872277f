// C ABI of the root-mean-square norm's gradients (rms_norm_backward.hpp): argument checks,
// launch shapes and launches.  The contract is stated in include/moe_decode.h.
#include "host.hpp"
#include "norm_shape.hpp"
#include "rms_norm_backward.hpp"

namespace {

using moe_host::aligned;
using moe_host::any_overlap;
using moe_host::rows_bytes;
using moe_host::rows_stride_ok;

size_t dtype_size(int dtype) { return dtype == MOE_F32 ? 4 : 2; }
bool dtype_ok(int dtype) { return dtype == MOE_F32 || dtype == MOE_BF16 || dtype == MOE_F16; }

int parts_of(int M) { return M < moe::kNormBackParts ? M : moe::kNormBackParts; }

// f<WR, P>(): wavefronts of a row and pieces of a lane, of which one leaves the registers for the next row's.  Two pieces
// spill 26 to 60 registers, four 347 to 489: bf16 with dsum, 8192 x 4096 55 us and 4096 x 8192 56 (4.8 TB/s), 2048 x 16384 95
// (2.8), 1024 x 32768 306 (0.9); columns beyond the row's end cost as much as those within (2047 x 16392 536).
template <typename F>
void by_row(int H, const F& f) {
  if (H <= 512) f.template operator()<1, 1>();
  else if (H <= 1024) f.template operator()<2, 1>();
  else if (H <= 2048) f.template operator()<4, 1>();
  else if (H <= 4096) f.template operator()<8, 1>();
  else if (H <= 8192) f.template operator()<16, 1>();
  else if (H <= 16384) f.template operator()<16, 2>();
  else f.template operator()<16, 4>();
}

template <typename T, typename W>
struct Backward {
  hipStream_t st;
  const void *dy, *r, *weight, *dsum;
  void* dx;
  const moe::NormBackwardArgs& a;
  int parts;
  template <int WR, int P>
  void operator()() const {
    hipLaunchKernelGGL((moe::rms_norm_backward_kernel<T, W, WR, P>), dim3((unsigned)parts),
                       dim3(moe::kNormBackThreads), 0, st, static_cast<const T*>(dy), static_cast<const T*>(r),
                       static_cast<const W*>(weight), static_cast<const T*>(dsum), static_cast<T*>(dx), a);
  }
};
template <typename T>
void launch(hipStream_t st, const void* dy, const void* r, const void* weight, bool f32_weight, const void* dsum, void* dx,
            const moe::NormBackwardArgs& a, int parts) {
  if (f32_weight) by_row(a.H, Backward<T, float>{st, dy, r, weight, dsum, dx, a, parts});
  else by_row(a.H, Backward<T, T>{st, dy, r, weight, dsum, dx, a, parts});
}

}  // namespace

extern "C" {

int moe_decode_rms_norm_backward_workspace(int M, int H, size_t* bytes) {
  const int rc = moe_host::check_norm(M, H);
  if (rc) return rc;
  if (!bytes) return MOE_ERR_NULL;
  *bytes = (size_t)parts_of(M) * H * 4;
  return MOE_OK;
}

int moe_decode_rms_norm_backward(const void* dy, long long ld_dy, const void* r, long long ld_r, int dtype,
                                 const void* weight, int weight_dtype, const float* rstd, const void* dsum,
                                 long long ld_dsum, void* dx, long long ld_dx, float* dweight, void* workspace,
                                 size_t workspace_bytes, int M, int H, void* stream) {
  const int rc = moe_host::check_norm(M, H);
  if (rc) return rc;
  if (!dtype_ok(dtype) || (weight_dtype != MOE_F32 && weight_dtype != dtype)) return MOE_ERR_ARG;
  if (M == 0) return MOE_OK;
  if (!rows_stride_ok(M, H, ld_dy) || !rows_stride_ok(M, H, ld_r) || (dsum && !rows_stride_ok(M, H, ld_dsum)) ||
      !rows_stride_ok(M, H, ld_dx))
    return MOE_ERR_SHAPE;
  if (!dy || !r || !weight || !rstd || !dx || !dweight || !workspace) return MOE_ERR_NULL;
  const size_t size = dtype_size(dtype);
  if (!aligned(dy, size) || !aligned(r, size) || !aligned(weight, dtype_size(weight_dtype)) || !aligned(rstd, 4) ||
      !aligned(dsum, size) || !aligned(dx, size) || !aligned(dweight, 4) || !aligned(workspace, 256))
    return MOE_ERR_ALIGN;
  const int parts = parts_of(M);
  const size_t need = (size_t)parts * H * 4;
  if (workspace_bytes < need) return MOE_ERR_ARG;
  const bool in_place = dsum == dx && (M <= 1 || ld_dsum == ld_dx);
  if (any_overlap({{dx, rows_bytes(M, H, ld_dx, size)}, {dweight, (size_t)H * 4}, {workspace, need}},
                  {{dy, rows_bytes(M, H, ld_dy, size)}, {r, rows_bytes(M, H, ld_r, size)},
                   {weight, (size_t)H * dtype_size(weight_dtype)}, {rstd, (size_t)M * 4},
                   {in_place ? nullptr : dsum, rows_bytes(M, H, ld_dsum, size)}}))
    return MOE_ERR_ALIAS;
  const moe::NormBackwardArgs a{ld_dy, ld_r, ld_dsum, ld_dx, rstd, static_cast<float*>(workspace), M, H};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const bool f = weight_dtype == MOE_F32;
  (void)hipGetLastError();
  if (dtype == MOE_F32) by_row(H, Backward<float, float>{st, dy, r, weight, dsum, dx, a, parts});
  else if (dtype == MOE_BF16) launch<__bf16>(st, dy, r, weight, f, dsum, dx, a, parts);
  else launch<moe::f16_t>(st, dy, r, weight, f, dsum, dx, a, parts);
  hipLaunchKernelGGL(moe::rms_norm_weight_kernel, dim3((unsigned)((H + 31) / 32)), dim3(moe::kNormSumThreads), 0, st, a.part,
                     dweight, parts, H);
  return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_LAUNCH;
}

}  // extern "C"
