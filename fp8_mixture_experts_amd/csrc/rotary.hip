// The norms of the heads of q and k with their rotation by position, and the
// gradients.
#include <hip/hip_runtime.h>

#include "block_util.h"
#include "rotary.h"

namespace mega_moe {

namespace {

constexpr int THREADS = 256;
constexpr double INV_2PI = 0.15915494309189533577;

// cos and sin of position * inv_freq, times scale.  The angle in turns is taken
// and reduced in float64 (a position of 10^6 has 10^5 turns, whose fraction
// float32 would leave 7 bits of); what is rounded is within half a turn.
__device__ __forceinline__ float2 turn(int position, float inv_freq, float scale) {
    const double turns = (double)position * (double)inv_freq * INV_2PI;
    float s, c;
    sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
    return float2{c * scale, s * scale};
}

// What the forward and the backward kernel have alike: a head is a row of D
// columns that LANES lanes hold, eight columns each, and the cos and sin of the
// workgroup's tokens lie in LDS, [token][R/2].
template <int LANES, typename Args>
struct Heads {
    const Args& a;
    const float2* cs;
    int col, j;                  // the lane's first column, and its place in the rotated part
    bool in, turned, second;     // second: of a pair's two columns, with the half layout

    __device__ Heads(const Args& a_, const float2* cs_) : a(a_), cs(cs_) {
        col = (threadIdx.x & (LANES - 1)) * 8;
        in = col < a.head_dim;
        j = col - a.rotary_start;
        turned = in && j >= 0 && j < a.rotary_dim;
        second = a.layout == MEGA_MOE_ROTARY_HALF && j >= a.rotary_dim / 2;
    }

    // The rotation of the lane's columns of token `t` of the workgroup's, or
    // its inverse (BACK).  All lanes of the wave call it.
    template <bool BACK>
    __device__ __forceinline__ void rotate(int t, float (&v)[8]) const {
        const float2* w = cs + t * (a.rotary_dim / 2);
        if (a.layout == MEGA_MOE_ROTARY_HALF) {
            const int half = a.rotary_dim / 16;          // lanes
            const int lane = threadIdx.x & 63, from = second ? lane - half : lane + half;
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __shfl(v[i], from & 63);
            if (!turned) return;
            w += second ? j - a.rotary_dim / 2 : j;
            const float sign = second != BACK ? 1.0f : -1.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = fmaf(v[i], w[i].x, sign * w[i].y * o[i]);
        } else if (turned) {
            w += j / 2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float x = v[2 * i], y = v[2 * i + 1], s = BACK ? -w[i].y : w[i].y;
                v[2 * i] = fmaf(x, w[i].x, -s * y);
                v[2 * i + 1] = fmaf(y, w[i].x, s * x);
            }
        }
    }
};

template <typename Args>
__device__ __forceinline__ void fill_turns(const Args& a, float2* cs, int64_t t0, int tokens) {
    const int half = a.rotary_dim / 2;
    const float scale = a.scale == 0.0f ? 1.0f : a.scale;
    for (int i = threadIdx.x; i < tokens * half; i += THREADS) {
        const int t = i / half;
        const int p = a.positions ? a.positions[t0 + t] : a.first_position + (int)(t0 + t);
        cs[i] = turn(p, a.inv_freq[i - t * half], scale);
    }
}

// LANES lanes hold a head of up to 8 LANES columns.
int lanes_of(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : 64; }

}  // namespace

// A workgroup takes `tokens` tokens and, of their heads, every gridDim.y-th
// round of 256 / LANES; q's heads come first, then k's.
template <bool F32, int LANES>
__global__ void __launch_bounds__(THREADS) moe_rotary(mega_moe_rotary_args a, int tokens) {
    extern __shared__ float2 turns[];
    constexpr int G = THREADS / LANES;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int n = (int)min((int64_t)tokens, a.num_tokens - t0);
    const int heads = a.q_heads + a.k_heads;
    const Heads<LANES, mega_moe_rotary_args> h(a, turns);
    float wq[8] = {}, wk[8] = {};
    if (h.in && a.q_weight) load8(a.q_weight, a.weight_type, h.col, wq);
    if (h.in && a.k_weight) load8(a.k_weight, a.weight_type, h.col, wk);
    fill_turns(a, turns, t0, n);
    __syncthreads();
    const float inv_d = 1.0f / (float)a.head_dim;
    for (int first = blockIdx.y * G; first < n * heads; first += gridDim.y * G) {
        const int item = first + threadIdx.x / LANES;
        const int t = item / heads, head = item - t * heads;
        const bool q = head < a.q_heads, live = item < n * heads && h.in;
        const int hh = q ? head : head - a.q_heads;
        float v[8] = {};
        if (live) {
            if (q) load8<F32>(a.q, (t0 + t) * a.q_stride + hh * a.q_head_stride + h.col, v);
            else load8<F32>(a.k, (t0 + t) * a.k_stride + hh * a.k_head_stride + h.col, v);
        }
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += v[i] * v[i];
        s = lanes_sum<LANES>(s);
        if (q ? a.q_weight != nullptr : a.k_weight != nullptr) {
            const float rs = rsqrtf(s * inv_d + a.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = v[i] * rs * (q ? wq[i] : wk[i]);
        }
        h.template rotate<false>(item < n * heads ? t : 0, v);
        if (live) {
            if (q) store8<F32>(a.q_out, (t0 + t) * a.q_out_stride + hh * a.q_out_head_stride + h.col, v);
            else store8<F32>(a.k_out, (t0 + t) * a.k_out_stride + hh * a.k_out_head_stride + h.col, v);
        }
    }
}

// Gradients: a workgroup goes from one run of tokens to the next and keeps its
// sums over tokens and heads, those of q and of k, in registers; at the end its
// groups meet in LDS and its sums go to the workspace, [grid][sums][D].
template <bool F32, int LANES>
__global__ void __launch_bounds__(THREADS) moe_rotary_backward(mega_moe_rotary_backward_args a, float* ws, int tokens) {
    extern __shared__ float2 turns[];
    constexpr int G = THREADS / LANES;
    const int heads = a.q_heads + a.k_heads;
    const Heads<LANES, mega_moe_rotary_backward_args> h(a, turns);
    float wq[8] = {}, wk[8] = {}, sq[8] = {}, sk[8] = {};
    if (h.in && a.q_weight) load8(a.q_weight, a.weight_type, h.col, wq);
    if (h.in && a.k_weight) load8(a.k_weight, a.weight_type, h.col, wk);
    const float inv_d = 1.0f / (float)a.head_dim;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.num_tokens; t0 += (int64_t)gridDim.x * tokens) {
        const int n = (int)min((int64_t)tokens, a.num_tokens - t0);
        fill_turns(a, turns, t0, n);
        __syncthreads();
        for (int first = 0; first < n * heads; first += G) {
            const int item = first + threadIdx.x / LANES;
            const int t = item / heads, head = item - t * heads;
            const bool q = head < a.q_heads, live = item < n * heads && h.in;
            const bool normed = q ? a.q_weight != nullptr : a.k_weight != nullptr;
            const int hh = q ? head : head - a.q_heads;
            float u[8] = {}, x[8] = {};
            if (live) {
                if (q) load8<F32>(a.dq_out, (t0 + t) * a.dq_out_stride + hh * a.dq_out_head_stride + h.col, u);
                else load8<F32>(a.dk_out, (t0 + t) * a.dk_out_stride + hh * a.dk_out_head_stride + h.col, u);
                if (normed) {
                    if (q) load8<F32>(a.q, (t0 + t) * a.q_stride + hh * a.q_head_stride + h.col, x);
                    else load8<F32>(a.k, (t0 + t) * a.k_stride + hh * a.k_head_stride + h.col, x);
                }
            }
            h.template rotate<true>(item < n * heads ? t : 0, u);
            float s = 0.0f, p = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s += x[i] * x[i];
                p += u[i] * (q ? wq[i] : wk[i]) * x[i];
            }
            s = lanes_sum<LANES>(s);
            p = lanes_sum<LANES>(p);
            if (normed) {
                const float rs = rsqrtf(s * inv_d + a.eps);
                const float mean = p * rs * inv_d;           // of u * weight * xh
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = x[i] * rs, g = u[i] * xh;
                    // a lane or a group that is out has u = 0, but xh may be infinite
                    if (live && q) sq[i] += g;
                    if (live && !q) sk[i] += g;
                    u[i] = rs * (u[i] * (q ? wq[i] : wk[i]) - xh * mean);
                }
            }
            if (live) {
                if (q) store8<F32>(a.dq, (t0 + t) * a.dq_stride + hh * a.dq_head_stride + h.col, u);
                else store8<F32>(a.dk, (t0 + t) * a.dk_stride + hh * a.dk_head_stride + h.col, u);
            }
        }
        __syncthreads();
    }
    // the groups' sums meet in LDS, in order
    __shared__ float part[G][LANES * 8];
    int k = 0;
    const auto put = [&](const float (&s)[8]) {
        store8<true>(&part[threadIdx.x / LANES][0], (size_t)(threadIdx.x & (LANES - 1)) * 8, s);
        __syncthreads();
        for (int c = threadIdx.x; c < a.head_dim; c += THREADS) {
            float o = 0.0f;
#pragma unroll
            for (int g = 0; g < G; ++g) o += part[g][c];
            ws[((size_t)blockIdx.x * rotary_sums(a) + k) * a.head_dim + c] = o;
        }
        __syncthreads();
        ++k;
    };
    if (a.dq_weight) put(sq);
    if (a.dk_weight) put(sk);
}

// Adds the workgroups' sums: a workgroup has 16 of the sums' columns, its 64
// groups of 16 lanes every 64th row each.
__global__ void __launch_bounds__(1024)
moe_rotary_reduce(const float* ws, float* out0, float* out1, int D, int sums, int rows) {
    __shared__ float part[64][17];
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int col = blockIdx.x * 16 + lane;              // of sums * D
    float s = 0.0f;
    if (col < sums * D) {
#pragma unroll 4
        for (int i = group; i < rows; i += 64) s += ws[(size_t)i * sums * D + col];
    }
    part[group][lane] = s;
    __syncthreads();
    if (group || col >= sums * D) return;
    s = 0.0f;
#pragma unroll
    for (int g = 0; g < 64; ++g) s += part[g][lane];
    if (col < D) out0[col] = s;
    else out1[col - D] = s;
}

namespace {

// Tokens of a workgroup at a time: what gives each of its threads a turn to work
// out, as long as that leaves a workgroup or more to every compute unit.
int tokens_of(int T, int R) {
    int n = R == 0 ? 8 : THREADS / (R / 2);
    if (n < 1) n = 1;
    if (n > 8) n = 8;
    while (n > 1 && (T + n - 1) / n < 1024) n /= 2;
    return n;
}

template <bool F32, typename Args, typename F>
void by_lanes(const Args& a, F go) {
    switch (lanes_of(a.head_dim)) {
        case 8: go(std::integral_constant<int, 8>()); break;
        case 16: go(std::integral_constant<int, 16>()); break;
        case 32: go(std::integral_constant<int, 32>()); break;
        default: go(std::integral_constant<int, 64>()); break;
    }
}

constexpr int BACKWARD_BLOCKS = 1024;

}  // namespace

void launch_rotary(const mega_moe_rotary_args& a, hipStream_t stream) {
    const int tokens = tokens_of(a.num_tokens, a.rotary_dim), G = THREADS / lanes_of(a.head_dim);
    const int blocks = (a.num_tokens + tokens - 1) / tokens;
    // few tokens: their heads over several workgroups
    const int rounds = (tokens * (a.q_heads + a.k_heads) + G - 1) / G;
    int split = (1024 + blocks - 1) / blocks;
    if (split > rounds) split = rounds;
    const unsigned lds = (unsigned)(tokens * a.rotary_dim * 4);
    const auto go = [&](auto f32) {
        by_lanes<decltype(f32)::value>(a, [&](auto lanes) {
            hipLaunchKernelGGL((moe_rotary<decltype(f32)::value, decltype(lanes)::value>), dim3((unsigned)blocks, (unsigned)split),
                               dim3(THREADS), lds, stream, a, tokens);
        });
    };
    if (a.type == MEGA_MOE_F32) go(std::true_type());
    else go(std::false_type());
}

int rotary_backward_blocks(const mega_moe_rotary_backward_args& a) {
    const int tokens = tokens_of(a.num_tokens, a.rotary_dim);
    const int need = (a.num_tokens + tokens - 1) / tokens;
    return need < BACKWARD_BLOCKS ? need : BACKWARD_BLOCKS;
}

void launch_rotary_backward(const mega_moe_rotary_backward_args& a, hipStream_t stream) {
    const int tokens = tokens_of(a.num_tokens, a.rotary_dim), blocks = rotary_backward_blocks(a);
    const unsigned lds = (unsigned)(tokens * a.rotary_dim * 4);
    float* ws = static_cast<float*>(a.workspace);
    if (blocks > 0) {
        const auto go = [&](auto f32) {
            by_lanes<decltype(f32)::value>(a, [&](auto lanes) {
                hipLaunchKernelGGL((moe_rotary_backward<decltype(f32)::value, decltype(lanes)::value>), dim3((unsigned)blocks),
                                   dim3(THREADS), lds, stream, a, ws, tokens);
            });
        };
        if (a.type == MEGA_MOE_F32) go(std::true_type());
        else go(std::false_type());
    }
    const int n = rotary_sums(a);
    if (n) {
        float* out0 = a.dq_weight ? a.dq_weight : a.dk_weight;
        hipLaunchKernelGGL(moe_rotary_reduce, dim3((unsigned)(n * a.head_dim + 15) / 16), dim3(1024), 0, stream, ws, out0,
                           n > 1 ? a.dk_weight : nullptr, a.head_dim, n, blocks);
    }
}

}  // namespace mega_moe
