// The router's selection and the gradient of its logits: one wave per token.
#include <hip/hip_runtime.h>

#include "router.h"
#include "router_row.h"

namespace mega_moe {

// The wave's largest key and the lowest index that has it.
template <typename Key>
__device__ __forceinline__ void wave_best(Key& key, int& idx) {
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
        const Key k2 = __shfl_xor(key, d, 64);
        const int i2 = __shfl_xor(idx, d, 64);
        if (k2 > key || (k2 == key && i2 < idx)) {
            key = k2;
            idx = i2;
        }
    }
}

constexpr int NO_EXPERT = 0x7fffffff;

// Key = float: order by the logits.  Key = double: order by score + bias.
template <int NI, typename Key>
__global__ void __launch_bounds__(256)
moe_router_topk(mega_moe_router_topk_args a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.num_tokens) return;
    const int E = a.num_experts, k = a.num_topk;
    int32_t* idx_out = a.topk_idx + (size_t)t * k;
    float* w_out = a.topk_weights + (size_t)t * k;
    if (a.token_mask && a.token_mask[t] == 0) {
        for (int j = lane; j < k; j += 64) {
            idx_out[j] = -1;
            w_out[j] = 0.0f;
        }
        return;
    }
    float l[NI], s[NI];
    load_row<NI>(a.logits, a.logits_type, (size_t)t * a.logits_stride, E, l);
    Key key[NI];
    if (a.score == MEGA_MOE_SCORE_SOFTMAX) {
        float top, sum;
        row_exp(l, s, top, sum);
        const float inv = 1.0f / sum;
#pragma unroll
        for (int i = 0; i < NI; ++i) s[i] *= inv;
        if constexpr (sizeof(Key) == 8) {
            double dsum = 0.0;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                key[i] = exp((double)l[i] - (double)top);
                dsum += key[i];
            }
            dsum = wave_sum(dsum);
#pragma unroll
            for (int i = 0; i < NI; ++i) key[i] /= dsum;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            s[i] = sigmoid(l[i]);
            if constexpr (sizeof(Key) == 8) key[i] = 1.0 / (1.0 + exp(-(double)l[i]));
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = i * 64 + lane;
        if constexpr (sizeof(Key) == 8) {
            if (a.bias && e < E) key[i] += (double)a.bias[e];
        } else {
            key[i] = l[i];
        }
        // never taken: -inf, NaN, and what lies behind the last expert
        if (!(l[i] > -INFINITY) || !(key[i] > (Key)-INFINITY)) key[i] = (Key)-INFINITY;
    }
    if constexpr (sizeof(Key) == 8) {
        if (a.num_groups > 1) {
            const int size = E / a.num_groups;
            double mine = -INFINITY;             // lane g holds group g's score
            for (int g = 0; g < a.num_groups; ++g) {
                double sum = 0.0;
                int first = NO_EXPERT;
                for (int r = 0; r < a.group_top; ++r) {
                    double best = -INFINITY;
                    int at = NO_EXPERT;
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        const int e = i * 64 + lane;
                        if (e >= g * size && e < (g + 1) * size && e != first && key[i] > best) {
                            best = key[i];
                            at = e;
                        }
                    }
                    wave_best(best, at);
                    sum += best;
                    first = at;
                }
                if (lane == g) mine = sum;
            }
            uint64_t kept = 0;
            for (int r = 0; r < a.topk_groups; ++r) {
                double best = lane < a.num_groups && !(kept >> lane & 1) ? mine : -INFINITY;
                int at = lane < a.num_groups && !(kept >> lane & 1) ? lane : NO_EXPERT;
                wave_best(best, at);
                if (at < 64) kept |= 1ull << at;     // none left: NaN scores
            }
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = i * 64 + lane;
                if (e < E && !(kept >> (e / size) & 1)) key[i] = -INFINITY;
            }
        }
    }
    // k rounds: the wave's best goes to lane j % 64, which writes it
    float total = 0.0f, mine_w = 0.0f;
    int mine_e = -1;
    for (int j = 0; j < k; ++j) {
        Key best = (Key)-INFINITY;
        int at = NO_EXPERT;
        float sc = 0.0f;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i * 64 + lane;
            }
        wave_best(best, at);
        const bool found = at != NO_EXPERT;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (at == i * 64 + lane) {
                sc = s[i];
                key[i] = (Key)-INFINITY;
            }
        sc = __shfl(sc, found ? at & 63 : 0, 64);
        if (!found) sc = 0.0f;
        total += sc;
        if ((j & 63) == lane) {
            mine_e = found ? at : -1;
            mine_w = sc;
            idx_out[j] = mine_e;
            if (k > 64) w_out[j] = mine_w;
        }
    }
    float scale = a.weight_scale;
    if (a.renormalize) scale = total == 0.0f ? 0.0f : scale / total;
    if (k <= 64) {
        if (lane < k) w_out[lane] = mine_w * scale;
    } else {
        for (int j = lane; j < k; j += 64) w_out[j] *= scale;
    }
}

// The sequence of token t: the last b with cu[b] <= t, if t < cu[b + 1]; -1 if
// there is none.  Empty sequences are passed over.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int B, int64_t t) {
    if (!cu) return 0;
    int lo = 0, hi = B;                      // cu[lo] <= t < cu[hi], if any
    if (t < cu[0] || t >= cu[B]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (cu[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

template <int NI>
__global__ void __launch_bounds__(256)
moe_router_backward(mega_moe_router_backward_args a) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= a.num_tokens) return;
    const int E = a.num_experts, k = a.num_topk;
    float* out = a.dlogits + (size_t)t * a.dlogits_stride;
    float d[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) d[i] = 0.0f;
    if (!a.token_mask || a.token_mask[t] != 0) {
        float l[NI], s[NI], ex[NI];
        load_row<NI>(a.logits, a.logits_type, (size_t)t * a.logits_stride, E, l);
        float top, sum;
        row_exp(l, ex, top, sum);
        const bool softmax = a.score == MEGA_MOE_SCORE_SOFTMAX;
        const float inv = sum > 0.0f ? 1.0f / sum : sum;
#pragma unroll
        for (int i = 0; i < NI; ++i) s[i] = softmax ? ex[i] * inv : sigmoid(l[i]);
        if (a.dweights) {
            // the scores that were taken, summed, and their product with dw
            float total = 0.0f, dot = 0.0f;
            const int32_t* idx = a.topk_idx + (size_t)t * k;
            const float* dw = a.dweights + (size_t)t * k;
            for (int j = 0; j < k; ++j) {
                const int e = idx[j];
                const float g = dw[j];
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (e == i * 64 + lane && e < E) {
                        total += s[i];
                        dot += g * s[i];
                    }
            }
            total = wave_sum(total);
            dot = wave_sum(dot);
            const bool renorm = a.renormalize != 0;
            const float scale = renorm ? (total == 0.0f ? 0.0f : a.weight_scale / total) : a.weight_scale;
            const float mean = renorm && total != 0.0f ? dot / total : 0.0f;
            float ds[NI];
#pragma unroll
            for (int i = 0; i < NI; ++i) ds[i] = 0.0f;
            for (int j = 0; j < k; ++j) {
                const int e = idx[j];
                const float g = scale * (dw[j] - mean);
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (e == i * 64 + lane && e < E) ds[i] += g;
            }
            if (softmax) {
                float c = 0.0f;
#pragma unroll
                for (int i = 0; i < NI; ++i) c += ds[i] * s[i];
                c = wave_sum(c);
#pragma unroll
                for (int i = 0; i < NI; ++i) d[i] += s[i] * (ds[i] - c);
            } else {
#pragma unroll
                for (int i = 0; i < NI; ++i) d[i] += ds[i] * sigmoid_slope(l[i]);
            }
        }
        const int B = a.cu_seqlens ? a.num_sequences : 1;
        const int b = a.dloss ? sequence_of(a.cu_seqlens, B, t) : -1;
        if (b >= 0) {
            const int n_b = a.tokens[b], n = a.tokens[B], live = a.tokens[B + 1];
            const float nb = (float)max(n_b, 1);
            const float scale = a.dloss[0] * a.balance_coeff / ((float)max(live, 1) * nb) *
                                ((float)E / ((float)k * nb));
            float f[NI], den = 0.0f, c = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                const int e = i * 64 + lane;
                f[i] = e < E ? scale * (float)a.counts[(size_t)b * E + e] : 0.0f;
                den += s[i];
                c += s[i] * f[i];
            }
            den = softmax ? 1.0f : wave_sum(den);
            const float id = den > 0.0f ? 1.0f / den : den;
            c = wave_sum(c) * id;
            const float lse = a.dloss[1] * a.z_coeff * 2.0f / (float)max(n, 1) * row_lse(top, sum) * inv;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                d[i] += (f[i] - c) * (softmax ? s[i] : sigmoid_slope(l[i]) * id);
                if (a.z_coeff != 0.0f) d[i] += lse * ex[i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = i * 64 + lane;
        if (e < E) out[e] = d[i];
    }
}

namespace {
// The smallest instance that holds E experts.
template <typename F>
void by_experts(int E, F&& go) {
    if (E <= 64) go(std::integral_constant<int, 1>{});
    else if (E <= 128) go(std::integral_constant<int, 2>{});
    else if (E <= 256) go(std::integral_constant<int, 4>{});
    else if (E <= 512) go(std::integral_constant<int, 8>{});
    else go(std::integral_constant<int, 16>{});
}
}  // namespace

void launch_router_topk(const mega_moe_router_topk_args& a, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)a.num_tokens + 3) / 4));
    const bool wide = a.bias || a.num_groups > 1;
    by_experts(a.num_experts, [&](auto ni) {
        constexpr int NI = decltype(ni)::value;
        if (wide) hipLaunchKernelGGL((moe_router_topk<NI, double>), grid, dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((moe_router_topk<NI, float>), grid, dim3(256), 0, stream, a);
    });
}

void launch_router_backward(const mega_moe_router_backward_args& a, hipStream_t stream) {
    const dim3 grid((unsigned)(((int64_t)a.num_tokens + 3) / 4));
    by_experts(a.num_experts, [&](auto ni) {
        constexpr int NI = decltype(ni)::value;
        hipLaunchKernelGGL((moe_router_backward<NI>), grid, dim3(256), 0, stream, a);
    });
}

}  // namespace mega_moe
