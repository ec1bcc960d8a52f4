// Launches of the router's selection, its losses and their gradients
// (router.hip, balance.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "mega_moe.h"

namespace mega_moe {

constexpr int ROUTER_MAX_GROUPS = 64;

void launch_router_topk(const mega_moe_router_topk_args& a, hipStream_t stream);
void launch_router_backward(const mega_moe_router_backward_args& a, hipStream_t stream);

int64_t balance_loss_workspace(const mega_moe_balance_loss_args& a);
void launch_balance_loss(const mega_moe_balance_loss_args& a, hipStream_t stream);

}  // namespace mega_moe
