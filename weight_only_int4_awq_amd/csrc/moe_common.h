// Shared by the kernels of mixture-of-experts layers (moe_route.hip) and of
// linears with an epilogue (linear_act.hip).
#pragma once

#include "awq_common.h"
#include "awq_internal.h"
#include "kv8_common.h"

namespace awq {

// Largest over the lanes of a wave, in every lane.
__device__ __forceinline__ uint32_t lanes_max(uint32_t x) {
#define AWQ_LANES_MAX(CTRL, ROWS)                                                                      \
  {                                                                                                    \
    const uint32_t o_ = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROWS, 0xf, true);       \
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
