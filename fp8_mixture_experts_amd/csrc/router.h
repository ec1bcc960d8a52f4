// Launches of the router's selection, its losses and their gradients
// (router.hip, balance.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "mega_moe.h"

namespace mega_moe {

constexpr int ROUTER_MAX_GROUPS = 64;

void launch_router_topk(const mega_moe_router_topk_args& a, hipStream_t stream);
void launch_router_backward(const mega_moe_router_backward_args& a, hipStream_t stream);

// Workgroups of the balance loss's second launch, of 256 threads each where there
// are many: a launch has fewer than 2^32 threads.
constexpr int BALANCE_SLICE = 32;             // experts per workgroup
constexpr int64_t BALANCE_MAX_GROUPS = (1 << 24) - 1;
inline int64_t balance_finish_groups(int64_t sequences, int64_t experts) {
    return sequences * ((experts + BALANCE_SLICE - 1) / BALANCE_SLICE);
}

int64_t balance_loss_workspace(const mega_moe_balance_loss_args& a);
void launch_balance_loss(const mega_moe_balance_loss_args& a, hipStream_t stream);

}  // namespace mega_moe
