// Sizes of the root-mean-square norm, shared by rms_norm.hip and
// rms_norm_backward.hip.
#pragma once

#include "moe_decode.h"

namespace moe_host {

constexpr int kNormMaxH = 32768;

// Threads of a pass: 64 a row up to 1024 columns, 256 up to 16384, else 1024, fewer than 2^32.
inline int check_norm(int M, int H) {
  if (M < 0 || H <= 0 || H > kNormMaxH || M >= (H <= 1024 ? 1 << 26 : H <= 16384 ? 1 << 24 : 1 << 22)) return MOE_ERR_SHAPE;
  return MOE_OK;
}

}  // namespace moe_host
