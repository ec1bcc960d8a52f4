// One token's logits in LANES neighbouring lanes (16, 32 or 64): lane l
// holds experts l, l + LANES, ...
#pragma once

#include "block_util.h"

namespace mega_moe {

template <int NI, int LANES = 64>
__device__ __forceinline__ void load_row(const void* logits, int type, size_t row, int E, float (&l)[NI]) {
    const int lane = threadIdx.x & (LANES - 1);
    const auto load = [&](auto index) {
        if (type == MEGA_MOE_F32) {
            const float* p = static_cast<const float*>(logits) + row;
#pragma unroll
            for (int i = 0; i < NI; ++i) l[i] = p[index(i)];
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(logits) + row;
#pragma unroll
            for (int i = 0; i < NI; ++i) l[i] = bf16_value(p[index(i)]);
        }
    };
    if (E == NI * LANES) {
        load([&](int i) { return i * LANES + lane; });
        return;
    }
    // lanes behind the last expert read it once more and drop it: no branches
    // between the loads
    load([&](int i) { return min(i * LANES + lane, E - 1); });
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

// Sums of scores below this are too small for their quotients: the reciprocals get
// near float32's largest value, and the scores subnormal or 0.  It means that every
// logit in the sum is below -55, where 1 + exp(logit) is 1 in float32: sigmoids are
// there in the proportions of exp(logit - largest logit), whose sum is 1 or more.
constexpr float SMALL_SUM = 0x1p-80f;

// The hardware reciprocal is within one step of the quotient, and its argument
// is at least 1.
__device__ __forceinline__ float sigmoid(float x) { return __builtin_amdgcn_rcpf(1.0f + expf(-x)); }

// Below it 1 + exp(x) is 1 in float32.
constexpr float LOW_LOGIT = -60.0f;

// sigmoid(x) and its derivative, from exp(-|x|): s (1 - s) would cancel where s
// is near 1.  With a `shift` below LOW_LOGIT that x does not pass, and `one` 0,
// both are exp(x - shift): the sigmoid and its derivative over the sigmoid of shift.
__device__ __forceinline__ void sigmoid_slope(float x, float& s, float& slope, float shift = 0.0f, float one = 1.0f) {
    const float e = expf(-fabsf(x - shift)), d = __builtin_amdgcn_rcpf(fmaf(e, one, 1.0f));
    s = x >= 0.0f ? d : e * d;
    slope = e * d * d;
}

// The sequence of token t: the last b with cu[b] <= t, if t < cu[b + 1]; -1 if
// there is none.  Empty sequences are passed over.
template <int LANES>
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int64_t t) {
    if (!cu) return 0;
    const int lane = threadIdx.x & (LANES - 1);
    if (B <= 2 * LANES) {
        // how many sequences end at t or before: loads that do not wait for each other
        int n = 0;
        for (int b = lane; b < B; b += LANES) n += cu[b + 1] <= t;
        n = (int)over_lanes<LANES>((uint32_t)n, [](uint32_t x, uint32_t y) { return x + y; });
        return t < cu[0] || n >= B ? -1 : n;
    }
    int lo = 0, hi = B;                      // cu[lo] <= t < cu[hi], if any
    if (t < cu[0] || t >= cu[B]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

}  // namespace mega_moe
