// The router's selection and the gradient of its logits.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "router.h"
#include "router_row.h"

namespace mega_moe {

constexpr int NO_EXPERT = 0x7fffffff;

// ---------------------------------------------------------------------------
// Selection.  A token's experts lie in 16 lanes (up to 256 experts, four tokens
// to a wave), in 32 (512) or in a wave.  k rounds each find the largest key and the lowest
// index that has it, by moves between lanes.  What bounds it is that chain of
// vector instructions: a token's logits are read once and are small.
//
// Without bias and groups the keys are the logits, which order the experts as
// the scores do.  Otherwise the order is that of score + bias in float64, but
// it is found in float32 first, with one round more than there are slots: a
// float32 score is off by less than `close` (below), so where any two
// neighbours of the order lie further apart than both their errors, the order
// is the float64 one.  Nearer ones (in one token of some hundreds) are ordered
// again by their float64 keys, one candidate to a lane; where that is not
// enough (softmax, whose float64 sum takes every expert; a near tie of groups,
// or of three at the last slot; more slots than lanes) the token goes through
// exact_topk, which computes all of it in float64.
// ---------------------------------------------------------------------------

// The score as a key: hardware exp2 and reciprocal.
__device__ __forceinline__ float sigmoid_key(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.44269504f));
}

// A bound on the error of a float32 key c = score + bias, in half steps of 1
// (2^-24).  Sigmoid: the exponent's two roundings and exp2's step move the
// score by s (1 - s) (2.9 |x| + 2) < 1.2, the sum by 1, the reciprocal by 2,
// the bias by |c|: less than 4.2 + |c|.
// Softmax: the rounding of l - max moves a score by at most 0.4 half steps of
// the largest one, the sum over lanes and exp by less than 40 of its own.
__device__ __forceinline__ float key_error(float c, bool softmax, float largest) {
    return 0x1p-23f * fabsf(c) + (softmax ? 0x1p-18f * largest : 0x1.4p-22f);
}

// The wave's largest key and the lowest index that has it (NO_EXPERT: none is
// above -inf).
template <int NI>
__device__ __forceinline__ int wave_best(const double (&key)[NI], double& best) {
    const int lane = threadIdx.x & 63;
    best = key[0];
#pragma unroll
    for (int i = 1; i < NI; ++i) best = fmax(best, key[i]);
    best = wave_max(best);
    if (!(best > -(double)INFINITY)) return NO_EXPERT;
    uint32_t at = NO_EXPERT;
#pragma unroll
    for (int i = NI - 1; i >= 0; --i)
        if (key[i] == best) at = i * 64 + lane;
    return (int)lanes_min<64>(at);
}

// The selection of token t in float64, by a whole wave: slots j, j + 64, ...
// of idx_out are written by lane j.  `kept`: the groups that stay, or 0 where
// float32 could not tell them either.
template <int NI>
__device__ __forceinline__ void exact_topk(const mega_moe_router_topk_args& a, int64_t t, uint64_t kept,
                                           int32_t* idx_out) {
    const int lane = threadIdx.x & 63, E = a.num_experts;
    float l[NI];
    double key[NI];
    load_row<NI>(a.logits, a.logits_type, (size_t)t * a.logits_stride, E, l);
    if (a.score == MEGA_MOE_SCORE_SOFTMAX) {
        float top = l[0];
#pragma unroll
        for (int i = 1; i < NI; ++i) top = fmaxf(top, l[i]);
        top = wave_max(top);
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            key[i] = exp((double)l[i] - (double)top);
            sum += key[i];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int i = 0; i < NI; ++i) key[i] /= sum;
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) key[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = i * 64 + lane;
        if (a.bias && e < E) key[i] += (double)a.bias[e];
        // never taken: -inf, NaN, and what lies behind the last expert
        if (!(l[i] > -INFINITY) || !(key[i] > -(double)INFINITY)) key[i] = -INFINITY;
    }
    if (a.num_groups > 1) {
        const int size = E / a.num_groups;
        if (kept == 0) {
            double mine[1] = {-INFINITY};        // lane g holds group g's score
            for (int g = 0; g < a.num_groups; ++g) {
                double of[NI], sum = 0.0;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    const int e = i * 64 + lane;
                    of[i] = e >= g * size && e < (g + 1) * size ? key[i] : -(double)INFINITY;
                }
                for (int r = 0; r < a.group_top; ++r) {
                    double best;
                    const int at = wave_best(of, best);
                    sum += best;
#pragma unroll
                    for (int i = 0; i < NI; ++i)
                        if (at == i * 64 + lane) of[i] = -INFINITY;
                }
                if (lane == g) mine[0] = sum;
            }
            for (int r = 0; r < a.topk_groups; ++r) {
                double best;
                int at = wave_best(mine, best);
                // only groups at -inf are left: the lowest of them
                if (at == NO_EXPERT) at = __builtin_ctzll(~kept);
                kept |= 1ull << at;
                if (lane == at) mine[0] = -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            const int e = i * 64 + lane;
            if (e < E && !(kept >> (e / size) & 1)) key[i] = -INFINITY;
        }
    }
    for (int j = 0; j < a.num_topk; ++j) {
        double best;
        const int at = wave_best(key, best);
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (at == i * 64 + lane) key[i] = -INFINITY;
        if ((j & 63) == lane) idx_out[j] = at != NO_EXPERT ? at : -1;
    }
}

// The two largest of the lanes' pairs first >= second.
template <int LANES>
__device__ __forceinline__ void lanes_top2(float& first, float& second) {
    const auto join = [&](uint32_t f1, uint32_t s1, uint32_t f2, uint32_t s2) {
        const float a = __uint_as_float(f1), b = __uint_as_float(f2);
        second = fmaxf(fminf(a, b), fmaxf(__uint_as_float(s1), __uint_as_float(s2)));
        first = fmaxf(a, b);
    };
    const auto f = [&] { return __float_as_uint(first); };
    const auto s = [&] { return __float_as_uint(second); };
    join(f(), s(), lane_pair<1>(f()), lane_pair<1>(s()));
    join(f(), s(), lane_pair<2>(f()), lane_pair<2>(s()));
    join(f(), s(), lane_pair<4>(f()), lane_pair<4>(s()));
    join(f(), s(), lane_pair<8>(f()), lane_pair<8>(s()));
    if constexpr (LANES >= 32) {
        const auto x = __builtin_amdgcn_permlane16_swap(f(), f(), false, false);
        const auto y = __builtin_amdgcn_permlane16_swap(s(), s(), false, false);
        join(x[0], y[0], x[1], y[1]);
    }
    if constexpr (LANES == 64) {
        const auto x = __builtin_amdgcn_permlane32_swap(f(), f(), false, false);
        const auto y = __builtin_amdgcn_permlane32_swap(s(), s(), false, false);
        join(x[0], y[0], x[1], y[1]);
    }
}

// SCORED: the keys are score + bias, else the logits.
template <int LANES, int NI, bool SCORED>
__global__ void __launch_bounds__(256)
moe_router_topk(mega_moe_router_topk_args a) {
    constexpr int ROWS = 64 / LANES;             // tokens per wave
    __shared__ float s_key[SCORED ? 4 * ROWS : 1][LANES * NI];
    __shared__ float s_group[SCORED ? 4 * ROWS : 1][ROUTER_MAX_GROUPS];
    const int lane = threadIdx.x & (LANES - 1), row = threadIdx.x / LANES;
    const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + row;
    const bool softmax = a.score == MEGA_MOE_SCORE_SOFTMAX;
    const int E = a.num_experts, k = a.num_topk;
    // rows that have nothing to do keep their lanes in step with the others
    const bool in = t < a.num_tokens;
    const bool live = in && (!a.token_mask || a.token_mask[t] != 0);
    if (__builtin_amdgcn_ballot_w64(in) == 0) return;
    const size_t at_row = (size_t)t * a.logits_stride;
    float l[NI], key[NI];
    if (live) {
        load_row<NI, LANES>(a.logits, a.logits_type, at_row, E, l);
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) l[i] = -INFINITY;
    }
    // the softmax of a score: exp(l - top) * inv
    float top = 0.0f, sum = 1.0f;
    if (softmax) row_exp<LANES>(l, key, top, sum);
    const float inv = 1.0f / sum;
    const float largest = softmax ? inv : 1.0f;      // of the scores
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int e = i * LANES + lane;
        if constexpr (SCORED) {
            key[i] = softmax ? key[i] * inv : sigmoid_key(l[i]);
            if (a.bias && e < E) key[i] += a.bias[e];
            // NaN, -inf, and what lies behind the last expert
            if (!(l[i] > -INFINITY) || !(key[i] > -INFINITY)) key[i] = -INFINITY;
        } else {
            key[i] = l[i] > -INFINITY ? l[i] : -INFINITY;
        }
    }
    bool near = false;
    uint64_t groups_kept = 0;
    if constexpr (SCORED) {
        if (a.num_groups > 1) {
            const int G = a.num_groups, size = E / G;
            float* groups = s_group[row];
            if (size % LANES == 0) {
                // whole rounds of the lanes: the two largest by moves
                float first = -INFINITY, second = -INFINITY;
                int g = 0, left = size;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    if (i * LANES >= E) break;
                    second = fmaxf(second, fminf(first, key[i]));
                    first = fmaxf(first, key[i]);
                    if ((left -= LANES) > 0) continue;
                    lanes_top2<LANES>(first, second);
                    if (lane == 0) groups[g] = a.group_top == 2 ? first + second : first;
                    first = second = -INFINITY;
                    left = size;
                    ++g;
                }
            } else {
                // through LDS, a lane per group; each starts elsewhere in its
                // group, so that the lanes read different banks
                float* keys = s_key[row];
#pragma unroll
                for (int i = 0; i < NI; ++i) keys[i * LANES + lane] = key[i];
                __builtin_amdgcn_wave_barrier();
                for (int g = lane; g < G; g += LANES) {
                    float first = -INFINITY, second = -INFINITY;
                    int o = g % size;
#pragma unroll 4
                    for (int j = 0; j < size; ++j) {
                        const float x = keys[g * size + o];
                        second = fmaxf(second, fminf(first, x));
                        first = fmaxf(first, x);
                        if (++o == size) o = 0;
                    }
                    groups[g] = a.group_top == 2 ? first + second : first;
                }
            }
            __builtin_amdgcn_wave_barrier();
            uint64_t kept = 0;
            float low = INFINITY, high = -INFINITY;      // the last one kept, the first one not
            for (int g0 = 0; g0 < G; g0 += LANES) {
                const int g = g0 + lane;
                bool keep = false;
                if (g < G) {
                    const float x = groups[g];
                    int before = 0;
                    for (int h = 0; h < G; ++h) {
                        const float y = groups[h];
                        before += y > x || (y == x && h < g);
                    }
                    keep = before < a.topk_groups;
                    if (keep) low = fminf(low, x);
                    else high = fmaxf(high, x);
                }
                const uint64_t b = __builtin_amdgcn_ballot_w64(keep);
                if constexpr (LANES == 64) kept = b;
                else kept |= (b >> ((threadIdx.x & 63) - lane) & ((1ull << (LANES & 63)) - 1)) << g0;
            }
            low = -lanes_max<LANES>(-low);
            high = lanes_max<LANES>(high);
            float widest = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (key[i] > -INFINITY) widest = fmaxf(widest, fabsf(key[i]));
            const float error = key_error(lanes_max<LANES>(widest), softmax, largest);
            near = high > -INFINITY && !(low - high > 8.0f * error);
            groups_kept = near ? 0 : kept;
            const uint32_t mul = ((1u << 20) + size - 1) / size;     // e / size for e * size < 2^20
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (!(kept >> ((uint32_t)(i * LANES + lane) * mul >> 20 & 63) & 1)) key[i] = -INFINITY;
        }
    }
    // the rounds; slot j belongs to lane j % LANES.  One more candidate than
    // slots, and another to see whether that one has near ties
    const int rounds = SCORED ? (k + 2 < E ? k + 2 : E) : k;
    const bool one_each = k < LANES;             // every candidate has a lane
    int32_t* idx_out = a.topk_idx + (size_t)t * k;
    float before = 0.0f;
    int mine = -1;
    bool tie = false, tie_at_k = false, full = near;
    for (int j = 0; j < rounds; ++j) {
        float best = key[0];
#pragma unroll
        for (int i = 1; i < NI; ++i) best = fmaxf(best, key[i]);
        best = lanes_max<LANES>(best);
        uint32_t at = NO_EXPERT;
#pragma unroll
        for (int i = NI - 1; i >= 0; --i)
            if (key[i] == best) at = i * LANES + lane;
        at = lanes_min<LANES>(at);
        const bool found = best > -INFINITY;
#pragma unroll
        for (int i = 0; i < NI; ++i)
            if (at == (uint32_t)(i * LANES + lane)) key[i] = -INFINITY;
        if constexpr (SCORED) {
            const bool close = j > 0 && found && !(before - best > 2.0f * key_error(before, softmax, largest));
            if (j <= k) tie = tie || close;
            if (j == k) tie_at_k = close;
            if (j == k + 1) full = full || (close && tie_at_k);
            before = best;
        }
        if ((j & (LANES - 1)) == lane && (j < k || (one_each && j == k))) {
            mine = found ? (int)at : -1;
            if (!one_each && in) idx_out[j] = mine;
        }
    }
    const auto logit = [&](int e) {
        return a.logits_type == MEGA_MOE_F32 ? static_cast<const float*>(a.logits)[at_row + e]
                                             : bf16_value(static_cast<const uint16_t*>(a.logits)[at_row + e]);
    };
    if constexpr (SCORED) {
        const bool by_lane = one_each && !softmax;
        if (!by_lane) full = full || tie;
        if (by_lane && __builtin_amdgcn_ballot_w64(tie) != 0) {
            // candidates by their float64 keys; those without an expert last
            const bool cand = lane <= k && mine >= 0;
            double c = -INFINITY;
            if (cand) c = 1.0 / (1.0 + exp(-(double)logit(mine))) + (a.bias ? (double)a.bias[mine] : 0.0);
            const int order = cand ? mine : NO_EXPERT - LANES + lane;
            int rank = 0;
            for (int i = 0; i <= k; ++i) {
                const double ci = __shfl(c, i, LANES);
                const int oi = __shfl(order, i, LANES);
                rank += ci > c || (ci == c && oi < order);
            }
            // lanes behind the candidates stay where they are
            if (lane > k) rank = lane;
            mine = __builtin_amdgcn_ds_permute((int)(((threadIdx.x & 63) - lane + rank) * 4), mine);
        }
        if (one_each && in && lane < k) idx_out[lane] = mine;
        // the whole wave on each token that needs all of it
        const uint64_t again = __builtin_amdgcn_ballot_w64(full && live);
        if (again) {
            const int64_t t0 = t - (threadIdx.x & 63) / LANES;
#pragma unroll 1
            for (int r = 0; r < ROWS; ++r) {
                const uint64_t mask = LANES == 64 ? ~0ull : ((1ull << (LANES & 63)) - 1) << (r * LANES);
                if (!(again & mask)) continue;
                const uint64_t kept = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(groups_kept >> 32), r * LANES) << 32 |
                                      (uint32_t)__builtin_amdgcn_readlane((int)groups_kept, r * LANES);
                exact_topk<(LANES * NI + 63) / 64>(a, t0 + r, kept, a.topk_idx + (size_t)(t0 + r) * k);
            }
            __threadfence_block();
            if (live && one_each && lane < k) mine = idx_out[lane];
        }
    } else {
        if (one_each && in && lane < k) idx_out[lane] = mine;
    }
    // the weights of the slots, from their own logits
    if (!in) return;
    float* w_out = a.topk_weights + (size_t)t * k;
    const auto score_of = [&](int e) {
        if (e < 0) return 0.0f;
        const float x = logit(e);
        return softmax ? expf(x - top) * inv : sigmoid(x);
    };
    float w = 0.0f, total = 0.0f;
    if (one_each) {
        if (lane < k) total = w = score_of(mine);
    } else {
        for (int j = lane; j < k; j += LANES) {
            w = score_of(idx_out[j]);
            w_out[j] = w;
            total += w;
        }
    }
    total = lanes_sum<LANES>(total);
    float scale = a.weight_scale;
    if (a.renormalize) scale = total == 0.0f ? 0.0f : scale / total;
    if (one_each) {
        if (lane < k) w_out[lane] = w * scale;
    } else {
        for (int j = lane; j < k; j += LANES) w_out[j] *= scale;
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

// The gradient of a token's logits, its experts in 16, 32 or 64 lanes.
template <int LANES, int NI>
__global__ void __launch_bounds__(256)
moe_router_backward(mega_moe_router_backward_args a) {
    const int lane = threadIdx.x & (LANES - 1);
    const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    if (t >= a.num_tokens) return;
    const int E = a.num_experts, k = a.num_topk;
    float* out = a.dlogits + (size_t)t * a.dlogits_stride;
    float d[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) d[i] = 0.0f;
    if (!a.token_mask || a.token_mask[t] != 0) {
        float l[NI], s[NI], ex[NI];
        load_row<NI, LANES>(a.logits, a.logits_type, (size_t)t * a.logits_stride, E, l);
        float top, sum;
        row_exp<LANES>(l, ex, top, sum);
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
                    if (e == i * LANES + lane && e < E) {
                        total += s[i];
                        dot += g * s[i];
                    }
            }
            total = lanes_sum<LANES>(total);
            dot = lanes_sum<LANES>(dot);
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
                    if (e == i * LANES + lane && e < E) ds[i] += g;
            }
            if (softmax) {
                float c = 0.0f;
#pragma unroll
                for (int i = 0; i < NI; ++i) c += ds[i] * s[i];
                c = lanes_sum<LANES>(c);
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
                const int e = i * LANES + lane;
                f[i] = e < E ? scale * (float)a.counts[(size_t)b * E + e] : 0.0f;
                den += s[i];
                c += s[i] * f[i];
            }
            den = softmax ? 1.0f : lanes_sum<LANES>(den);
            const float id = den > 0.0f ? 1.0f / den : den;
            c = lanes_sum<LANES>(c) * id;
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
        const int e = i * LANES + lane;
        if (e < E) out[e] = d[i];
    }
}

namespace {
// The smallest instance that holds E experts.
template <typename F>
void by_experts(int E, F&& go) {
    using std::integral_constant;
    if (E <= 16) go(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    else if (E <= 32) go(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    else if (E <= 64) go(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    else if (E <= 128) go(integral_constant<int, 16>{}, integral_constant<int, 8>{});
    else if (E <= 256) go(integral_constant<int, 16>{}, integral_constant<int, 16>{});
    else if (E <= 512) go(integral_constant<int, 32>{}, integral_constant<int, 16>{});
    else go(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}
unsigned workgroups(int tokens, int lanes) { return (unsigned)(((int64_t)tokens * lanes + 255) / 256); }
}  // namespace

void launch_router_topk(const mega_moe_router_topk_args& a, hipStream_t stream) {
    const bool scored = a.bias || a.num_groups > 1;
    by_experts(a.num_experts, [&](auto lanes, auto ni) {
        constexpr int L = decltype(lanes)::value, NI = decltype(ni)::value;
        const dim3 grid(workgroups(a.num_tokens, L));
        if (scored) hipLaunchKernelGGL((moe_router_topk<L, NI, true>), grid, dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((moe_router_topk<L, NI, false>), grid, dim3(256), 0, stream, a);
    });
}

void launch_router_backward(const mega_moe_router_backward_args& a, hipStream_t stream) {
    by_experts(a.num_experts, [&](auto lanes, auto ni) {
        constexpr int L = decltype(lanes)::value, NI = decltype(ni)::value;
        hipLaunchKernelGGL((moe_router_backward<L, NI>), dim3(workgroups(a.num_tokens, L)), dim3(256), 0, stream, a);
    });
}

}  // namespace mega_moe
