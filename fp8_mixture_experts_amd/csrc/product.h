// Launches of the E4M3 product (product.hip) and what the host plans for it.
#pragma once

#include <hip/hip_runtime.h>

#include "mega_moe.h"

namespace mega_moe {

// Bytes of partial sums that a call puts into its workspace.
int64_t product_workspace(int m, int n, int k, int b_scale, int out_type);

void launch_product(const mega_moe_product_args& a, hipStream_t stream);

}  // namespace mega_moe
