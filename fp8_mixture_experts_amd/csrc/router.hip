// The router's selection and the gradient of its logits.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "router.h"
#include "router_row.h"

namespace mega_moe {

constexpr int NO_EXPERT = 0x7fffffff;

// ---------------------------------------------------------------------------
// Selection.  A token's experts lie in 16, 32 or 64 lanes; k rounds each find
// the largest key and the lowest index that has it, by moves between lanes.  For
// more than a few rounds the lanes sort their keys first.  What bounds it is that
// chain of vector instructions: a token's logits are read once and are small.
// 8192 tokens of 256 experts, k = 8: the logits' order 7.6 us a call; sigmoid with a
// bias 8.2, in 8 groups too 10.8 (the 8.5 MB that it has to move: 1.7 us).  How many
// near ones turn up goes by the data (below): softmax in 8 groups 14 us from float32
// logits and 23 from BF16 ones, sigmoid with a bias in 8 groups 11 from either.
//
// Without bias and groups the keys are the logits, which order the experts as
// the scores do.  Otherwise the order is that of score + bias in float64, but
// it is found in float32 first, with one round more than there are slots: a
// float32 score is off by less than `close` (below), so where any two
// neighbours of the order lie further apart than both their errors, the order
// is the float64 one.  Nearer ones (in one token of some hundreds with float32
// logits; BF16 ones are often equal: without a bias, over 8 groups, a third of the
// tokens have two such among their first nine of 256 experts) are ordered again by
// their float64 keys, one candidate to a lane; where that is not enough (softmax, whose
// float64 sum takes every expert; three near ones at the last slot; more slots than
// lanes) the token goes through exact_topk, a whole wave to one token after another,
// which computes all of it in float64.  Groups with near scores, likewise, are
// ordered by exact_groups.
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

// The float64 keys of token t, its experts over a whole wave.
template <int NI>
__device__ __forceinline__ void exact_keys(const mega_moe_router_topk_args& a, int64_t t, double (&key)[NI]) {
    const int lane = threadIdx.x & 63, E = a.num_experts;
    float l[NI];
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
        if (a.bias) key[i] += (double)a.bias[min(i * 64 + lane, E - 1)];
        // never taken: -inf, NaN, and what lies behind the last expert
        if (!(l[i] > -INFINITY) || !(key[i] > -(double)INFINITY)) key[i] = -INFINITY;
    }
}

// The groups of token t that stay: those of `sure`, and `need` of `maybe`, the
// ones that float32 cannot tell apart, by their float64 scores.
template <int NI>
__device__ __forceinline__ uint64_t exact_groups(const mega_moe_router_topk_args& a, int64_t t, uint64_t sure,
                                                 uint64_t maybe, int need) {
    const int lane = threadIdx.x & 63, size = a.num_experts / a.num_groups;
    double key[NI], mine[1] = {-INFINITY};       // lane g holds group g's score
    exact_keys<NI>(a, t, key);
    for (uint64_t rest = maybe; rest != 0; rest &= rest - 1) {
        const int g = __builtin_ctzll(rest);
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
    for (int r = 0; r < need; ++r) {
        double best;
        int at = wave_best(mine, best);
        // only groups at -inf are left: the lowest of them
        if (at == NO_EXPERT) at = __builtin_ctzll(maybe & ~sure);
        sure |= 1ull << at;
        if (lane == at) mine[0] = -INFINITY;
    }
    return sure;
}

// The selection of token t among the groups `kept` in float64, by a whole
// wave: slots j, j + 64, ... of idx_out are written by lane j.
template <int NI>
__device__ __forceinline__ void exact_topk(const mega_moe_router_topk_args& a, int64_t t, uint64_t kept,
                                           int32_t* idx_out) {
    const int lane = threadIdx.x & 63, E = a.num_experts;
    double key[NI];
    exact_keys<NI>(a, t, key);
    if (a.num_groups > 1) {
        const int size = E / a.num_groups;
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

__device__ __forceinline__ uint64_t of_lane(uint64_t v, int lane) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((int)v, lane);
}

// The two largest of N values each over 16 lanes, N <= 16 a power of two.  Every
// step joins a lane with another one, of the other half of what is left; while
// there are several values each of the two goes on with half of them.  The
// result of value i is in the lanes whose upper bits are i.
template <int D, int N, bool FIRST, int M>
__device__ __forceinline__ void top2_step(float (&first)[M], float (&second)[M]) {
    constexpr int H = N > 1 ? N / 2 : 1;
    const bool up = (threadIdx.x & D) != 0;
    const auto pair = [](float v) { return __uint_as_float(lane_pair<D>(__float_as_uint(v))); };
#pragma unroll
    for (int j = 0; j < H; ++j) {
        constexpr int O = N > 1 ? H : 0;
        const float f = up ? first[j + O] : first[j], f2 = pair(up ? first[j] : first[j + O]);
        if constexpr (FIRST) {
            second[j] = fminf(f, f2);
        } else {
            const float s = up ? second[j + O] : second[j], s2 = pair(up ? second[j] : second[j + O]);
            second[j] = fmaxf(fminf(f, f2), fmaxf(s, s2));
        }
        first[j] = fmaxf(f, f2);
    }
}

template <int N>
__device__ __forceinline__ void top2_of_16(float (&first)[N], float (&second)[N]) {
    const auto left = [](int n) constexpr { return N / n > 1 ? N / n : 1; };
    top2_step<8, left(1), true>(first, second);
    top2_step<4, left(2), false>(first, second);
    top2_step<2, left(4), false>(first, second);
    top2_step<1, left(8), false>(first, second);
}

// A lane's keys in order, the largest first and, with BY_INDEX, equal ones by
// index, by merging neighbours R apart.
template <int N, bool BY_INDEX>
struct Sorted {
    float key[N];
    int at[N];
    template <int A, int B>
    __device__ __forceinline__ void order() {
        const bool swap = key[B] > key[A] || (BY_INDEX && key[B] == key[A] && at[B] < at[A]);
        const float k = swap ? key[B] : key[A];
        const int i = swap ? at[B] : at[A];
        key[B] = swap ? key[A] : key[B];
        at[B] = swap ? at[A] : at[B];
        key[A] = k;
        at[A] = i;
    }
    template <int LO, int LEN, int R, int I>
    __device__ __forceinline__ void order_from() {
        if constexpr (I + R < LO + LEN) {
            order<I, I + R>();
            order_from<LO, LEN, R, I + 2 * R>();
        }
    }
    template <int LO, int LEN, int R>
    __device__ __forceinline__ void merge() {
        if constexpr (2 * R < LEN) {
            merge<LO, LEN, 2 * R>();
            merge<LO + R, LEN, 2 * R>();
            order_from<LO, LEN, R, LO + R>();
        } else {
            order<LO, LO + R>();
        }
    }
    template <int LO, int LEN>
    __device__ __forceinline__ void sort() {
        if constexpr (LEN > 1) {
            sort<LO, LEN / 2>();
            sort<LO + LEN / 2, LEN / 2>();
            merge<LO, LEN, 1>();
        }
    }
};

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
    if constexpr (SCORED) {
        float bias[NI];
#pragma unroll
        for (int i = 0; i < NI; ++i) bias[i] = 0.0f;
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < NI; ++i) bias[i] = a.bias[min(i * LANES + lane, E - 1)];
        }
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            key[i] = (softmax ? key[i] * inv : sigmoid_key(l[i])) + bias[i];
            // NaN, -inf, and what lies behind the last expert
            key[i] = l[i] > -INFINITY && key[i] > -INFINITY ? key[i] : -INFINITY;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) key[i] = l[i] > -INFINITY ? l[i] : -INFINITY;
    }
    uint64_t kept = 0;
    if constexpr (SCORED) {
        if (a.num_groups > 1) {
            const int G = a.num_groups, size = E / G;
            float* groups = s_group[row];
            if (size % 16 == 0) {
                // the two largest of every 16 experts, then a lane per group
                float first[NI], second[NI];
#pragma unroll
                for (int i = 0; i < NI; ++i) first[i] = key[i];
                top2_of_16<NI>(first, second);
                f32x2_t* of = reinterpret_cast<f32x2_t*>(s_key[row]);
                constexpr int SAME = 16 / NI;            // lanes with the same result
                if (lane % SAME == 0)
                    of[lane % 16 / SAME * (LANES / 16) + lane / 16] = f32x2_t{first[0], second[0]};
                __builtin_amdgcn_wave_barrier();
                for (int g = lane; g < G; g += LANES) {
                    f32x2_t m = of[g * (size / 16)];
                    for (int j = 1; j < size / 16; ++j) {
                        const f32x2_t o = of[g * (size / 16) + j];
                        m[1] = fmaxf(fminf(m[0], o[0]), fmaxf(m[1], o[1]));
                        m[0] = fmaxf(m[0], o[0]);
                    }
                    groups[g] = a.group_top == 2 ? m[0] + m[1] : m[0];
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
            // each group's place among them, by counting
            const auto row_bits = [&](bool v) {
                const uint64_t b = __builtin_amdgcn_ballot_w64(v) >> ((threadIdx.x & 63) - lane);
                return LANES == 64 ? b : b & ((1ull << (LANES & 63)) - 1);
            };
            float low = INFINITY, high = -INFINITY;      // the last one kept, the first one not
            for (int g0 = 0; g0 < G; g0 += LANES) {
                const int g = g0 + lane;
                bool keep = false;
                if (g < G) {
                    const float x = groups[g];
                    int place = 0;
                    for (int h = 0; h < G; ++h) {
                        const float y = groups[h];
                        place += y > x || (y == x && h < g);
                    }
                    keep = place < a.topk_groups;
                    if (keep) low = fminf(low, x);
                    else high = fmaxf(high, x);
                }
                kept |= row_bits(keep) << g0;
            }
            low = -lanes_max<LANES>(-low);
            high = lanes_max<LANES>(high);
            float widest = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i)
                if (key[i] > -INFINITY) widest = fmaxf(widest, fabsf(key[i]));
            // a group's score is off by three errors of its largest key at most
            const float margin = 6.0f * key_error(lanes_max<LANES>(widest), softmax, largest);
            const bool near = live && high > -INFINITY && !(low - high > margin);
            const uint64_t again = __builtin_amdgcn_ballot_w64(near);
            if (again) {
                uint64_t maybe = 0;
                for (int g0 = 0; g0 < G; g0 += LANES) {
                    const float x = g0 + lane < G ? groups[g0 + lane] : -INFINITY;
                    maybe |= row_bits(g0 + lane < G && !(x > low + margin) && !(x < high - margin)) << g0;
                }
                const uint64_t sure = kept & ~maybe;
                const int need = a.topk_groups - __builtin_popcountll(sure);
                const int64_t t0 = t - (threadIdx.x & 63) / LANES;
#pragma unroll 1
                for (int r = 0; r < ROWS; ++r) {
                    if (!(again >> (r * LANES) & 1)) continue;
                    const uint64_t k2 = exact_groups<(LANES * NI + 63) / 64>(
                        a, t0 + r, of_lane(sure, r * LANES), of_lane(maybe, r * LANES),
                        __builtin_amdgcn_readlane(need, r * LANES));
                    if ((threadIdx.x & 63) / LANES == r) kept = k2;
                }
            }
            const uint32_t mul = ((1u << 20) + size - 1) / size;     // e / size for e * size < 2^20
            if (G <= 32) {
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (!__builtin_amdgcn_ubfe((uint32_t)kept, (uint32_t)(i * LANES + lane) * mul >> 20, 1)) key[i] = -INFINITY;
            } else {
#pragma unroll
                for (int i = 0; i < NI; ++i)
                    if (!(kept >> ((uint32_t)(i * LANES + lane) * mul >> 20 & 63) & 1)) key[i] = -INFINITY;
            }
        }
    }
    // The rounds; slot j belongs to lane j % LANES.  With scores one candidate
    // more than slots is found, and another to see whether that one has near
    // ties; each has a lane, or all of it is left to exact_topk.
    const bool one_each = SCORED ? k + 2 <= LANES : k <= LANES;
    const int rounds = !SCORED ? k : !one_each ? 0 : k + 2 < E ? k + 2 : E;
    int32_t* idx_out = a.topk_idx + (size_t)t * k;
    float c = -INFINITY;
    int mine = -1;
    const auto take = [&](int j, float best, uint32_t at) {
        if ((j & (LANES - 1)) != lane) return;
        c = best;
        mine = best > -INFINITY ? (int)at : -1;
        if (!SCORED && !one_each && in) idx_out[j] = mine;
    };
    // The lanes' keys in order, so that a round looks at their heads alone: pays
    // from NI / 2 rounds on.  8192 tokens, 256 experts: one round 4.4 us without
    // and 5.2 with, eight 7.3 and 6.7; 32768 of 1024: one 30 and 43, eight 67 and 63.
    if (rounds > NI / 2) {
        // equal scores are ordered with the near ones below
        Sorted<NI, !SCORED> mem;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            mem.key[i] = key[i];
            mem.at[i] = i;
        }
        mem.template sort<0, NI>();
        using Order = std::conditional_t<(NI > 8), uint64_t, uint32_t>;
        Order order = 0;                         // four bits to a key
#pragma unroll
        for (int i = 0; i < NI; ++i) order |= (Order)mem.at[i] << (4 * i);
        for (int j = 0; j < rounds; ++j) {
            const float best = lanes_max<LANES>(mem.key[0]);
            const uint32_t here =
                mem.key[0] == best ? (uint32_t)order % 16 * LANES + (uint32_t)lane : (uint32_t)NO_EXPERT;
            const uint32_t at = lanes_min<LANES>(here);
            const bool gone = at == here;
#pragma unroll
            for (int i = 0; i + 1 < NI; ++i) mem.key[i] = gone ? mem.key[i + 1] : mem.key[i];
            mem.key[NI - 1] = gone ? -INFINITY : mem.key[NI - 1];
            order = gone ? order >> 4 : order;
            take(j, best, at);
        }
    } else {
        for (int j = 0; j < rounds; ++j) {
            float best = key[0];
#pragma unroll
            for (int i = 1; i < NI; ++i) best = fmaxf(best, key[i]);
            best = lanes_max<LANES>(best);
            int first = NI;                      // this lane's first key that is the best
#pragma unroll
            for (int i = NI - 1; i >= 0; --i) first = key[i] == best ? i : first;
            const uint32_t here = first < NI ? (uint32_t)(first * LANES + lane) : (uint32_t)NO_EXPERT;
            const uint32_t at = lanes_min<LANES>(here);
            const int gone = at == here ? first : -1;
#pragma unroll
            for (int i = 0; i < NI; ++i) key[i] = gone == i ? -INFINITY : key[i];
            take(j, best, at);
        }
    }
    const auto logit = [&](int e) {
        return a.logits_type == MEGA_MOE_F32 ? static_cast<const float*>(a.logits)[at_row + e]
                                             : bf16_value(static_cast<const uint16_t*>(a.logits)[at_row + e]);
    };
    // the logits of the candidates: for their weights, and to tell near ones apart
    float x = one_each && mine >= 0 ? logit(mine) : 0.0f;
    if constexpr (SCORED) {
        // which candidates are too close to the next one to be told apart
        const float next = __shfl_down(c, 1, LANES);
        const bool close = lane <= k && next > -INFINITY && !(c - next > 2.0f * key_error(c, softmax, largest));
        const uint64_t b = __builtin_amdgcn_ballot_w64(close) >> ((threadIdx.x & 63) - lane);
        const bool tie = one_each && (b & ((1ull << k) - 1)) != 0;
        const bool three_at_k = one_each && (b >> (k - 1) & 3) == 3;
        const bool full = !one_each || (tie && (softmax || three_at_k));
        if (!softmax && __builtin_amdgcn_ballot_w64(tie) != 0) {
            // candidates by their float64 keys; those without an expert last
            const bool cand = lane <= k && mine >= 0;
            double d = -INFINITY;
            if (cand) d = 1.0 / (1.0 + exp(-(double)x)) + (a.bias ? (double)a.bias[mine] : 0.0);
            const int order = cand ? mine : NO_EXPERT - LANES + lane;
            int rank = 0;
            for (int i = 0; i <= k; ++i) {
                const double di = __shfl(d, i, LANES);
                const int oi = __shfl(order, i, LANES);
                rank += di > d || (di == d && oi < order);
            }
            // lanes behind the candidates stay where they are
            if (lane > k) rank = lane;
            const int to = (int)(((threadIdx.x & 63) - lane + rank) * 4);
            mine = __builtin_amdgcn_ds_permute(to, mine);
            x = __int_as_float(__builtin_amdgcn_ds_permute(to, __float_as_int(x)));
        }
        if (one_each && in && lane < k) idx_out[lane] = mine;
        if (!one_each && in && !live)
            for (int j = lane; j < k; j += LANES) idx_out[j] = -1;
        // the whole wave on each token that needs all of it
        const uint64_t again = __builtin_amdgcn_ballot_w64(full && live);
        if (again) {
            const int64_t t0 = t - (threadIdx.x & 63) / LANES;
#pragma unroll 1
            for (int r = 0; r < ROWS; ++r) {
                const uint64_t mask = LANES == 64 ? ~0ull : ((1ull << (LANES & 63)) - 1) << (r * LANES);
                if (!(again & mask)) continue;
                exact_topk<(LANES * NI + 63) / 64>(a, t0 + r, of_lane(kept, r * LANES),
                                                    a.topk_idx + (size_t)(t0 + r) * k);
            }
            __threadfence_block();
            if (live && one_each && lane < k) {
                mine = idx_out[lane];
                x = mine >= 0 ? logit(mine) : 0.0f;
            }
        }
    } else {
        if (one_each && in && lane < k) idx_out[lane] = mine;
    }
    // the weights of the slots, from their own logits
    if (!in) return;
    float* w_out = a.topk_weights + (size_t)t * k;
    // the score, or its proportion to that of the logit `most`
    bool small = false;
    float most = -INFINITY;
    const auto score_of = [&](int e, float l) {
        if (e < 0) return 0.0f;
        if (small) return expf(l - most);
        if (softmax) return expf(l - top) * inv;
        // 1 + exp(l) is 1, and what the reciprocal would flush to 0 a subnormal
        return l < -64.0f ? expf(l) : sigmoid(l);
    };
    float w = 0.0f, total = 0.0f;
    const auto slots = [&](auto&& f) {
        if (one_each) {
            if (lane < k) f(lane, mine, x);
        } else {
            for (int j = lane; j < k; j += LANES) {
                const int e = idx_out[j];
                f(j, e, e >= 0 ? logit(e) : 0.0f);
            }
        }
    };
    const auto score_slots = [&] {
        total = 0.0f;
        slots([&](int j, int e, float l) {
            w = score_of(e, l);
            if (!one_each) w_out[j] = w;
            total += w;
        });
        total = lanes_sum<LANES>(total);
    };
    score_slots();
    float scale = a.weight_scale;
    if (a.renormalize) {
        if (total < SMALL_SUM) {
            // Only their proportions are asked for.  Where no score is above 2^-80 they
            // are those of exp(logit), of a softmax always.
            slots([&](int, int e, float l) { most = e >= 0 ? fmaxf(most, l) : most; });
            most = lanes_max<LANES>(most);
            small = most > -INFINITY;
            if (small) score_slots();
        }
        scale = total == 0.0f ? 0.0f : scale / total;
    }
    // a quotient beyond float32, though the weights are not
    const bool apart = isinf(scale);
    const auto scaled = [&](float w) { return apart ? w / total * a.weight_scale : w * scale; };
    if (one_each) {
        if (lane < k) w_out[lane] = scaled(w);
    } else {
        for (int j = lane; j < k; j += LANES) w_out[j] = scaled(w_out[j]);
    }
}

// The gradient of a token's logits, its experts in 16, 32 or 64 lanes.  The
// top-k weights reach the scores that were taken (one slot to a lane, added to
// the row through LDS); softmax spreads minus their mean over all experts.
// Bound by memory for large batches (32768 tokens of 256 experts from the weights
// 15.8 us, 4.4 TB/s, for sigmoids 14.0, 5.0 TB/s; with the losses 20 and 23), by a
// token's chain of loads and sums for others: 8192 tokens 6.3, 5.1, 7.4 and 8.7 us.
template <int LANES, int NI>
__global__ void __launch_bounds__(256)
moe_router_backward(mega_moe_router_backward_args a) {
    __shared__ float s_row[256 / LANES][LANES * NI];
    const int lane = threadIdx.x & (LANES - 1);
    const int64_t t = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
    if (t >= a.num_tokens) return;
    const int E = a.num_experts, k = a.num_topk;
    float* out = a.dlogits + (size_t)t * a.dlogits_stride;
    float d[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) d[i] = 0.0f;
    if (!a.token_mask || a.token_mask[t] != 0) {
        const bool softmax = a.score == MEGA_MOE_SCORE_SOFTMAX;
        const bool z = a.dloss && a.z_coeff != 0.0f;
        const size_t at_row = (size_t)t * a.logits_stride;
        const int B = a.cu_seqlens ? a.num_sequences : 1;
        const int b = a.dloss ? sequence_of<LANES>(a.cu_seqlens, B, t) : -1;
        float l[NI], s[NI], slope[NI], ex[NI], top = 0.0f, sum = 1.0f;
        load_row<NI, LANES>(a.logits, a.logits_type, at_row, E, l);
        if (softmax || z) row_exp<LANES>(l, ex, top, sum);
        const float inv = sum > 0.0f ? 1.0f / sum : sum;
        // The losses see the sigmoids' proportions alone: of a row without a logit above
        // LOW_LOGIT those of exp(logit - largest), whose sum has a reciprocal.
        float most = -INFINITY;
        if (!softmax && b >= 0) {
            most = top;
            if (!z) {
                most = l[0];
#pragma unroll
                for (int i = 1; i < NI; ++i) most = fmaxf(most, l[i]);
                most = lanes_max<LANES>(most);
            }
        }
        const bool low = most < LOW_LOGIT && most > -INFINITY;
        const float shift = low ? most : 0.0f, one = low ? 0.0f : 1.0f;
        if (softmax || b >= 0) {                 // the weights' gradient alone has no use for other sigmoids
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                if (softmax) s[i] = slope[i] = ex[i] * inv;
                else sigmoid_slope(l[i], s[i], slope[i], shift, one);
            }
        }
        if (a.dweights) {
            const int32_t* idx = a.topk_idx + (size_t)t * k;
            const float* dw = a.dweights + (size_t)t * k;
            float* row = s_row[threadIdx.x / LANES];
            // rounds of LANES slots: first their scores' sum and its product
            // with dw, then the slots' parts of the gradient
            float ref = softmax ? top : 0.0f, fac = softmax ? inv : 1.0f, most_taken = -INFINITY;
            const auto slot = [&](int j, int& e, float& g, float& sj, float& slj) {
                e = j < k ? idx[j] : -1;
                g = sj = slj = 0.0f;
                if (e < 0 || e >= E) {
                    e = -1;
                    return;
                }
                g = dw[j];
                const float x = a.logits_type == MEGA_MOE_F32
                                    ? static_cast<const float*>(a.logits)[at_row + e]
                                    : bf16_value(static_cast<const uint16_t*>(a.logits)[at_row + e]);
                most_taken = fmaxf(most_taken, x);
                if (softmax) sj = slj = expf(x - ref) * fac;
                else sigmoid_slope(x, sj, slj, ref, fac);
            };
            int e;
            float g, sj, slj, total, dot;
            const bool renorm = a.renormalize != 0;
            for (bool again = renorm;;) {
                total = dot = 0.0f;
                for (int j0 = 0; j0 < k; j0 += LANES) {
                    slot(j0 + lane, e, g, sj, slj);
                    total += sj;
                    dot += g * sj;
                }
                total = lanes_sum<LANES>(total);
                dot = lanes_sum<LANES>(dot);
                if (!again || !(total < SMALL_SUM)) break;
                // Once more, relative to the largest of them: only the proportions count,
                // and those of the sigmoids' slopes are the same, since 1 - s is 1.
                ref = lanes_max<LANES>(most_taken);
                if (ref == -INFINITY) break;
                fac = softmax ? 1.0f : 0.0f;
                again = false;
            }
            // the factor of a slot's slope, and weight_scale apart: their product may be
            // beyond float32 where the gradients are not
            const float part = !renorm ? 1.0f : total == 0.0f ? 0.0f : 1.0f / total;
            const float mean = renorm ? dot * part : 0.0f;
            float c = 0.0f;
            for (int j0 = 0; j0 < k; j0 += LANES) {
                if (k > LANES) slot(j0 + lane, e, g, sj, slj);
                const float v = e >= 0 ? a.weight_scale * ((g - mean) * (slj * part)) : 0.0f;
                c += v;
                // an expert taken twice: found by who wrote last
                if (e >= 0) row[e] = __int_as_float(lane);
                __builtin_amdgcn_wave_barrier();
                const bool lost = e >= 0 && __float_as_int(row[e]) != lane;
                const bool twice = lanes_max<LANES>(lost ? 1.0f : 0.0f) != 0.0f;
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = 0; i < NI; ++i) row[i * LANES + lane] = 0.0f;
                __builtin_amdgcn_wave_barrier();
                if (!twice) {
                    if (e >= 0) row[e] = v;
                } else {
                    for (int j = 0; j < LANES; ++j) {
                        if (lane == j && e >= 0) row[e] += v;
                        __builtin_amdgcn_wave_barrier();
                    }
                }
                __builtin_amdgcn_wave_barrier();
#pragma unroll
                for (int i = 0; i < NI; ++i) d[i] += row[i * LANES + lane];
                __builtin_amdgcn_wave_barrier();
            }
            if (softmax) {
                c = lanes_sum<LANES>(c);
#pragma unroll
                for (int i = 0; i < NI; ++i) d[i] -= c * s[i];
            }
        }
        if (b >= 0) {
            const int n_b = a.tokens[b], n = a.tokens[B], live = a.tokens[B + 1];
            const float nb = (float)max(n_b, 1);
            const float scale = a.dloss[0] * a.balance_coeff / ((float)max(live, 1) * nb) *
                                ((float)E / ((float)k * nb));
            const int32_t* counts = a.counts + (size_t)b * E;
            float f[NI], den = 0.0f, c = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) f[i] = scale * (float)counts[min(i * LANES + lane, E - 1)];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                den += s[i];
                c += s[i] * f[i];
            }
            den = softmax ? 1.0f : lanes_sum<LANES>(den);
            const float id = den > 0.0f ? 1.0f / den : den;
            c = lanes_sum<LANES>(c) * id;
            const float lse = z ? a.dloss[1] * a.z_coeff * 2.0f / (float)max(n, 1) * row_lse(top, sum) * inv : 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                d[i] += (f[i] - c) * slope[i] * id;
                if (z) d[i] += lse * ex[i];
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
template <int N>
using Int = std::integral_constant<int, N>;

template <typename F>
void by_experts(int E, int lanes, F&& go) {
    if (E <= 128 && lanes <= 16) {
        if (E <= 16) go(Int<16>{}, Int<1>{});
        else if (E <= 32) go(Int<16>{}, Int<2>{});
        else if (E <= 64) go(Int<16>{}, Int<4>{});
        else go(Int<16>{}, Int<8>{});
    } else if (E <= 256 && lanes <= 32) {
        if (E <= 64) go(Int<32>{}, Int<2>{});
        else if (E <= 128) go(Int<32>{}, Int<4>{});
        else go(Int<32>{}, Int<8>{});
    } else {
        if (E <= 64) go(Int<64>{}, Int<1>{});
        else if (E <= 128) go(Int<64>{}, Int<2>{});
        else if (E <= 256) go(Int<64>{}, Int<4>{});
        else if (E <= 512) go(Int<64>{}, Int<8>{});
        else go(Int<64>{}, Int<16>{});
    }
}

// Lanes per token (at least): fewer of them do less work in all, a step over lanes
// serving more tokens, but in a longer chain per wave.  The selection (k = 8) with
// 64, 32 and 16 lanes: 64 experts, 8192 tokens 7.3, 5.0 and 4.2 us; 128 experts,
// 1024 tokens 4.2, 4.5 and 4.9, 4096 6.1, 5.0 and 5.1, 8192 9.2, 6.3 and 5.7; 256
// experts, 1024 tokens 4.4, 5.0 and 5.7, 4096 6.2, 5.4 and 5.9, 8192 9.1, 6.9 and
// 6.9.  `slots` that each need a lane can ask for more.
int lanes_for(int E, int tokens, int slots) {
    const int lanes = E <= 64 || (E <= 128 && tokens > 4096) ? 16 : tokens > 2048 ? 32 : 64;
    return slots > 32 ? 64 : slots > lanes ? 32 : lanes;
}
unsigned workgroups(int tokens, int lanes) { return (unsigned)(((int64_t)tokens * lanes + 255) / 256); }
}  // namespace

void launch_router_topk(const mega_moe_router_topk_args& a, hipStream_t stream) {
    const bool scored = a.bias || a.num_groups > 1;
    const int slots = scored ? a.num_topk + 2 : a.num_topk;
    by_experts(a.num_experts, lanes_for(a.num_experts, a.num_tokens, slots), [&](auto lanes, auto ni) {
        constexpr int L = decltype(lanes)::value, NI = decltype(ni)::value;
        const dim3 grid(workgroups(a.num_tokens, L));
        if (scored) hipLaunchKernelGGL((moe_router_topk<L, NI, true>), grid, dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((moe_router_topk<L, NI, false>), grid, dim3(256), 0, stream, a);
    });
}

void launch_router_backward(const mega_moe_router_backward_args& a, hipStream_t stream) {
    by_experts(a.num_experts, lanes_for(a.num_experts, a.num_tokens, 0), [&](auto lanes, auto ni) {
        constexpr int L = decltype(lanes)::value, NI = decltype(ni)::value;
        hipLaunchKernelGGL((moe_router_backward<L, NI>), dim3(workgroups(a.num_tokens, L)), dim3(256), 0, stream, a);
    });
}

}  // namespace mega_moe
