// Launches of the E4M3 product (product.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "mega_moe.h"
#include "product_plan.h"

namespace mega_moe {

// Bytes of partial sums that a call puts into its workspace.
int64_t product_workspace(const ProductPlan& plan, int m, int n);

void launch_product(const mega_moe_product_args& a, const ProductPlan& plan, hipStream_t stream);

}  // namespace mega_moe
