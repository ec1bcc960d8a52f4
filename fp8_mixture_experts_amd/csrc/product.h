// Launches of the E4M3 product (product.hip) and what the host plans for it.
#pragma once

#include <hip/hip_runtime.h>

#include "mega_moe.h"

namespace mega_moe {

// The kernel and tile of a call, and the parts that its steps are split into.
struct ProductPlan {
    int kind, splits;
};
ProductPlan product_plan(int m, int n, int k, int out_type);

// Bytes of partial sums that a call puts into its workspace.
int64_t product_workspace(const ProductPlan& plan, int m, int n);

void launch_product(const mega_moe_product_args& a, const ProductPlan& plan, hipStream_t stream);

}  // namespace mega_moe
