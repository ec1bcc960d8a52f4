// Launches of the kernels that make the products' operands (quantize.hip).
#pragma once

#include <hip/hip_runtime.h>

#include "mega_moe.h"

namespace mega_moe {

void launch_quantize(const mega_moe_quantize_args& a, hipStream_t stream);
void launch_swiglu_backward(const mega_moe_swiglu_backward_args& a, hipStream_t stream);

}  // namespace mega_moe
