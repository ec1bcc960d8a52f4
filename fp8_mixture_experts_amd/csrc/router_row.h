// One token's logits in LANES neighbouring lanes (16, 32 or 64): lane l
// holds experts l, l + LANES, ...
#pragma once

#include "block_util.h"

namespace mega_moe {

template <int NI, int LANES = 64>
__device__ __forceinline__ void load_row(const void* logits, int type, size_t row, int E, float (&l)[NI]) {
    const int lane = threadIdx.x & (LANES - 1);
    // lanes behind the last expert read it once more and drop it: no branches
    // between the loads
    if (type == MEGA_MOE_F32) {
        const float* p = static_cast<const float*>(logits) + row;
#pragma unroll
        for (int i = 0; i < NI; ++i) l[i] = p[min(i * LANES + lane, E - 1)];
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(logits) + row;
#pragma unroll
        for (int i = 0; i < NI; ++i) l[i] = bf16_value(p[min(i * LANES + lane, E - 1)]);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) l[i] = i * LANES + lane < E ? l[i] : -INFINITY;
}

// The largest logit of the row, and the sum of exp(logit - largest).  A row of
// -inf alone has sum 0.  An infinity or NaN among the logits makes the sum NaN.
template <int LANES = 64, int NI>
__device__ __forceinline__ void row_exp(const float (&l)[NI], float (&ex)[NI], float& top, float& sum) {
    top = l[0];
#pragma unroll
    for (int i = 1; i < NI; ++i) top = fmaxf(top, l[i]);
    top = lanes_max<LANES>(top);
    const float at = top == -INFINITY ? 0.0f : top;
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        ex[i] = expf(l[i] - at);
        sum += ex[i];
    }
    sum = lanes_sum<LANES>(sum);
}

// log sum exp of the row; 0 for a row of -inf alone, so that a token without
// any expert adds nothing to a loss.
__device__ __forceinline__ float row_lse(float top, float sum) { return sum == 0.0f ? 0.0f : logf(sum) + top; }

__device__ __forceinline__ float sigmoid(float x) { return 1.0f / (1.0f + expf(-x)); }

// sigmoid(x) and its derivative, from exp(-|x|): s (1 - s) would cancel where s
// is near 1.
__device__ __forceinline__ void sigmoid_slope(float x, float& s, float& slope) {
    const float e = expf(-fabsf(x)), d = 1.0f / (1.0f + e);
    s = x >= 0.0f ? d : e * d;
    slope = e * d * d;
}

}  // namespace mega_moe
