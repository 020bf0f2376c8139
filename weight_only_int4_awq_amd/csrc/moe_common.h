// Shared by the kernels of mixture-of-experts layers (moe_route.hip) and of
// linears with an epilogue (linear_act.hip): sums over the lanes of a wave and
// the arguments of a product whose rows are grouped by expert.
#pragma once

#include "awq_common.h"
#include "awq_internal.h"

namespace awq {

// Inclusive sum over the lanes of a wave, in six register moves.
__device__ __forceinline__ int lanes_scan(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);   // lane - 1 of the row of 16
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);   // - 2
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);   // - 4
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);   // - 8
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);   // the row before's last
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);   // the half before's last
  return x;
}

// Largest over the lanes of a wave, in every lane.
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
#define AWQ_LANES_MAX(CTRL, ROWS)                                                                      \
  {                                                                                                    \
    const uint32_t o_ = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, false);      \
    x = x > o_ ? x : o_;                                                                               \
  }
  AWQ_LANES_MAX(0x111, 0xf)
  AWQ_LANES_MAX(0x112, 0xf)
  AWQ_LANES_MAX(0x114, 0xf)
  AWQ_LANES_MAX(0x118, 0xf)
  AWQ_LANES_MAX(0x142, 0xa)
  AWQ_LANES_MAX(0x143, 0xc)
#undef AWQ_LANES_MAX
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}

}  // namespace awq
