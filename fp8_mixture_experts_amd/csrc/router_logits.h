// Launches of the router product's kernels (router_logits.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "mega_moe.h"

namespace mega_moe {

int64_t router_logits_workspace(const mega_moe_router_logits_args& a);
void launch_router_logits(const mega_moe_router_logits_args& a, hipStream_t stream);
void launch_router_logits_backward(const mega_moe_router_logits_args& a, hipStream_t stream);

}  // namespace mega_moe
