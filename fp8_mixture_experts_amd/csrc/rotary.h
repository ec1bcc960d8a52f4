// Launches of the head norms with rotation (rotary.hip) and what the host plans
// for them.
#pragma once

#include <hip/hip_runtime.h>

#include "mega_moe.h"

namespace mega_moe {

// Weights' gradients, [D] each.
__host__ __device__ inline int rotary_sums(const mega_moe_rotary_backward_args& a) {
    return (a.dq_weight != nullptr) + (a.dk_weight != nullptr);
}

// Workgroups of the backward kernel, each with sums of its own.
int rotary_backward_blocks(const mega_moe_rotary_backward_args& a);

void launch_rotary(const mega_moe_rotary_args& a, hipStream_t stream);
void launch_rotary_backward(const mega_moe_rotary_backward_args& a, hipStream_t stream);

}  // namespace mega_moe
