// Scan over a wave, for the kernels that sort or look up by running counts.
#pragma once

#include <hip/hip_runtime.h>

namespace mx {

// Inclusive scan over the wave of values that are not negative: shifts inside
// the 16-lane rows, then each row's last lane to the rows after it.
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_or_zero(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
template <typename Op>
__device__ __forceinline__ int scan64(int v, Op op) {
  v = op(v, dpp_or_zero<0x111, 0xF>(v));
  v = op(v, dpp_or_zero<0x112, 0xF>(v));
  v = op(v, dpp_or_zero<0x114, 0xF>(v));
  v = op(v, dpp_or_zero<0x118, 0xF>(v));
  v = op(v, dpp_or_zero<0x142, 0xA>(v));
  v = op(v, dpp_or_zero<0x143, 0xC>(v));
  return v;
}

}  // namespace mx
