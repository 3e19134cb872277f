// Which form of the norm's kernels a row takes: the wavefronts of one row and the
// pieces of 8 columns of a lane, shared by rms_norm.hip and rms_norm_backward.hip.
#pragma once

#include "moe_decode.h"
#include "pieces.hpp"

namespace moe_host {

constexpr int kNormMaxH = 32768;

inline int check_norm(int M, int H) {
  if (M < 0 || H <= 0 || H > kNormMaxH || M >= (H <= 4096 ? 1 << 26 : H <= 16384 ? 1 << 24 : 1 << 22)) return MOE_ERR_SHAPE;
  return MOE_OK;   // threads: 64 a row up to 4096 columns, 256 up to 16384, else 1024, fewer than 2^32
}

// f<WR, P>(): one wavefront a row up to 4096 columns, 4 up to 16384, else 16.
template <typename F>
void by_row(int H, const F& f) {
  if (H <= 512) f.template operator()<1, 1>();
  else if (H <= 1024) f.template operator()<1, 2>();
  else if (H <= 2048) f.template operator()<1, 4>();
  else if (H <= 4096) f.template operator()<1, 8>();
  else if (H <= 8192) f.template operator()<4, 4>();
  else if (H <= 16384) f.template operator()<4, 8>();
  else f.template operator()<16, 4>();
}

}  // namespace moe_host
