// Launches of the norm kernels (norm.hip) and what the host plans for them.
#pragma once

#include <hip/hip_runtime.h>

#include "mega_moe.h"

namespace mega_moe {

// Gradients that are sums over the tokens, [H] each.
__host__ __device__ inline int norm_sums(const mega_moe_norm_backward_args& a) {
    return (a.dpre_weight != nullptr) + (a.dpost_weight != nullptr) +
           (a.gate_kind == MEGA_MOE_GATE_CHANNEL && a.dgate != nullptr);
}

// Workgroups of the backward kernel, each with sums of its own.
int norm_backward_blocks(int tokens, int hidden);

void launch_norm(const mega_moe_norm_args& a, hipStream_t stream);
void launch_norm_backward(const mega_moe_norm_backward_args& a, hipStream_t stream);

}  // namespace mega_moe
