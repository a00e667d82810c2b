// Host-side argument validation of the entry points of forge_ops.h. Pure C++,
// as validate.hpp. Order of checks: DTYPE, NULL, SHAPE, ALIGN, ALIAS,
// CLIP_NOT_FUSABLE, HPARAM, TILE.
#pragma once

#include <cstdint>

#include "forge_ops.h"
#include "validate.hpp"

namespace forge {

// Elements of all tensors of a list together: keeps the norm's chunk indexes
// within 31 bits.
constexpr int64_t kMaxListElems = int64_t(1) << 42;

int64_t grad_norm_workspace(int32_t count);
forge_status validate_grad_norm(const forge_tensor* tensors, int32_t count, double max_norm,
                                const float* norm_coef, const void* workspace,
                                int64_t workspace_bytes);
forge_status validate_clip_grads(const forge_tensor* tensors, int32_t count, const float* coef);
forge_status validate_adamw_clipped(const forge_tensor* tensors, int32_t count, const float* coef,
                                    const forge_adamw_params* p);
forge_status validate_sgdm_clipped(const forge_tensor* tensors, int32_t count, const float* coef,
                                   const forge_sgdm_params* p);

}  // namespace forge
