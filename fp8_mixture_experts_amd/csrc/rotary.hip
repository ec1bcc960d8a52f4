// The norms of the heads of q and k with their rotation by position, and the
// gradients.
#include <hip/hip_runtime.h>

#include "block_util.h"
#include "rotary.h"

namespace mega_moe {

namespace {

constexpr int THREADS = 256;             // of the forward kernel
constexpr int BACK_THREADS = 1024;       // of the backward kernel: few workgroups leave few sums
constexpr int BACK_BLOCKS = 256;         // one to a compute unit
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

// Of `tokens` tokens from t0 on, every by-th; `sign` is the angles'.
template <int NT, typename Args>
__device__ __forceinline__ void fill_turns(const Args& a, float2* cs, int t0, int by, int tokens, float sign = 1.0f) {
    const int half = a.rotary_dim / 2;
    const float scale = a.scale == 0.0f ? 1.0f : a.scale;
    for (int i = threadIdx.x; i < tokens * half; i += NT) {
        const int t = i / half;
        const int token = t0 + t * by;
        const int p = a.positions ? a.positions[token] : a.first_position + token;
        cs[i] = turn(p, a.inv_freq[i - t * half] * sign, scale);
    }
}

// One head of one token: a group's item, and the one `by` items on.
struct Item {
    int t, head, heads, by_t, by_head;
    __device__ Item(int first, int by, int heads_) : heads(heads_) {
        t = first / heads, head = first - t * heads;
        by_t = by / heads, by_head = by - by_t * heads;
    }
    __device__ __forceinline__ void next() {
        t += by_t, head += by_head;
        if (head >= heads) head -= heads, ++t;
    }
};

// A tensor of heads.
struct Rows {
    const void* p;
    int64_t token, head;
    __device__ __forceinline__ int64_t at(int64_t t, int h, int col) const { return t * token + h * head + col; }
};

// Eight columns as they lie in memory.
template <bool F32>
struct Raw {
    static constexpr int N = F32 ? 2 : 1;
    u32x4_t d[N];
    __device__ __forceinline__ void load(bool live, const Rows& rows, int64_t t, int head, int col) {
#pragma unroll
        for (int n = 0; n < N; ++n) d[n] = live ? raw8<F32>(rows.p, rows.at(t, head, col))[n] : u32x4_t{0u, 0u, 0u, 0u};
    }
    __device__ __forceinline__ void get(float (&v)[8]) const { values8<F32>(d, v); }
};

// LANES lanes hold a head of up to 8 LANES columns.
int lanes_of(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : D <= 256 ? 32 : 64; }

}  // namespace

// A workgroup takes `tokens` tokens and, of their heads, every gridDim.y-th
// round of 256 / LANES: q's, then k's.  Eight workgroups to a compute unit keep the
// memory busy: with the next round's loads in flight in each, whose registers
// leave room for seven, 49 us against 38 (8192 tokens of 32 + 8 heads of 128).
// That is 168 MB, 4.5 TB/s with the call (a copy's rate would be 33 us; 32768 tokens go at 5.2);
// one token takes the launch and its angles (6.6 us with the call, 3.3 the kernel).
template <bool F32, int LANES>
__global__ void __launch_bounds__(THREADS) moe_rotary(mega_moe_rotary_args a, int tokens, float sign) {
    extern __shared__ float2 turns[];
    constexpr int G = THREADS / LANES;
    const int t0 = blockIdx.x * tokens, n = min(tokens, a.num_tokens - t0), by = gridDim.y * G;
    const Heads<LANES, mega_moe_rotary_args> h(a, turns);
    fill_turns<THREADS>(a, turns, t0, 1, n, sign);
    __syncthreads();
    const float inv_d = 1.0f / (float)a.head_dim;
    const auto run = [&](int heads, const Rows& in, const Rows& out, const void* weight) {
        if (heads == 0) return;
        float w[8] = {};
        if (h.in && weight) load8(weight, a.weight_type, h.col, w);
        Item at(blockIdx.y * G + threadIdx.x / LANES, by, heads);
        for (int first = blockIdx.y * G; first < n * heads; first += by, at.next()) {
            const bool live = at.t < n && h.in;
            Raw<F32> raw;
            raw.load(live, in, t0 + at.t, at.head, h.col);
            float v[8], s = 0.0f;
            raw.get(v);
            if (weight) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s += v[i] * v[i];
                const float rs = rsqrtf(lanes_sum<LANES>(s) * inv_d + a.eps);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = v[i] * rs * w[i];
            }
            h.template rotate<false>(at.t < n ? at.t : 0, v);
            if (live) store8<F32>(const_cast<void*>(out.p), out.at(t0 + at.t, at.head, h.col), v);
        }
    };
    run(a.q_heads, Rows{a.q, a.q_stride, a.q_head_stride}, Rows{a.q_out, a.q_out_stride, a.q_out_head_stride}, a.q_weight);
    run(a.k_heads, Rows{a.k, a.k_stride, a.k_head_stride}, Rows{a.k_out, a.k_out_stride, a.k_out_head_stride}, a.k_weight);
}

// Gradients where there is a weight: a workgroup goes from one run of tokens to another (of their heads it
// takes every gridDim.y-th round).  Its sums over tokens and heads lie in LDS, a place
// for each thread, and in registers during a run; at the end the groups' meet
// in order and the workgroup's go to the workspace, [grid][sums][D].  The next round's loads
// are in flight over the two sums of a head; two rounds ahead, or the first loaded over the angles, was no faster.
// Memory bounds it, and the second launch: 4096 tokens of 32 + 8 heads of 128 32.3 us with the sums' (126 MB; a
// copy's rate would be 24.7, the second launch is 4), 16384 tokens 108 us (4.7 TB/s).
template <bool F32, int LANES>
__global__ void __launch_bounds__(BACK_THREADS) moe_rotary_backward(mega_moe_rotary_backward_args a, float* ws, int tokens) {
    extern __shared__ float2 turns[];
    constexpr int G = BACK_THREADS / LANES;
    __shared__ __attribute__((aligned(16))) float part[2][BACK_THREADS][8];
    const int by = gridDim.y * G;
    const Heads<LANES, mega_moe_rotary_backward_args> h(a, turns);
    const float inv_d = 1.0f / (float)a.head_dim;
    {
        const float zero[8] = {};
        store8<true>(part[0][threadIdx.x], 0, zero);
        store8<true>(part[1][threadIdx.x], 0, zero);
    }
    // A run has every gridDim.x-th token, so that the workgroups go through memory side by side (with
    // neighbours 16384 tokens of 32 + 8 heads of 128 took 114 us, not 108).
    const int between = gridDim.x;
    for (int t0 = blockIdx.x; t0 < a.num_tokens; t0 += between * tokens) {
        const int left = a.num_tokens - t0, n = left >= tokens * between ? tokens : (left + between - 1) / between;
        fill_turns<BACK_THREADS>(a, turns, t0, between, n);
        __syncthreads();
#pragma unroll 1
        for (int side = 0; side < 2; ++side) {
            const bool q = side == 0;
            const int heads = q ? a.q_heads : a.k_heads;
            if (heads == 0) continue;
            const Rows in = q ? Rows{a.q, a.q_stride, a.q_head_stride} : Rows{a.k, a.k_stride, a.k_head_stride};
            const Rows dout = q ? Rows{a.dq_out, a.dq_out_stride, a.dq_out_head_stride} : Rows{a.dk_out, a.dk_out_stride, a.dk_out_head_stride};
            const Rows dx = q ? Rows{a.dq, a.dq_stride, a.dq_head_stride} : Rows{a.dk, a.dk_stride, a.dk_head_stride};
            const void* weight = q ? a.q_weight : a.k_weight;
            float w[8] = {}, sum[8];
            if (h.in && weight) load8(weight, a.weight_type, h.col, w);
            load8<true>(part[side][threadIdx.x], 0, sum);
            Item at(blockIdx.y * G + threadIdx.x / LANES, by, heads);
            Raw<F32> raw_u, raw_x;
            const auto fetch = [&]() {
                const bool live = at.t < n && h.in;
                const int token = t0 + at.t * between;
                raw_u.load(live, dout, token, at.head, h.col);
                raw_x.load(live && weight, in, token, at.head, h.col);
            };
            fetch();
            for (int first = blockIdx.y * G; first < n * heads; first += by) {
                const int t = at.t, head = at.head;
                const bool live = t < n && h.in;
                float u[8], x[8];
                raw_u.get(u);
                raw_x.get(x);
                at.next();
                if (first + by < n * heads) fetch();
                h.template rotate<true>(t < n ? t : 0, u);
                if (weight) {
                    float s = 0.0f, p = 0.0f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        s += x[i] * x[i];
                        p += u[i] * w[i] * x[i];
                    }
                    const float rs = rsqrtf(lanes_sum<LANES>(s) * inv_d + a.eps);
                    const float mean = lanes_sum<LANES>(p) * rs * inv_d;     // of u * weight * xh
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float xh = x[i] * rs;
                        // a lane or a group that is out has u = 0, but xh may be infinite
                        if (live) sum[i] += u[i] * xh;
                        u[i] = rs * (u[i] * w[i] - xh * mean);
                    }
                }
                if (live) store8<F32>(const_cast<void*>(dx.p), dx.at(t0 + t * between, head, h.col), u);
            }
            store8<true>(part[side][threadIdx.x], 0, sum);
        }
        __syncthreads();
    }
    __syncthreads();
    for (int i = threadIdx.x; i < rotary_sums(a) * a.head_dim; i += BACK_THREADS) {
        const int k = i / a.head_dim, c = i - k * a.head_dim, side = a.dq_weight ? k : 1;
        float o = 0.0f;
#pragma unroll 16
        for (int g = 0; g < G; ++g) o += part[side][g * LANES + c / 8][c & 7];
        ws[(size_t)(blockIdx.y * gridDim.x + blockIdx.x) * rotary_sums(a) * a.head_dim + i] = o;
    }
}

// Adds the workgroups' sums (atomics would add them in an order that changes): a workgroup has 16 of the
// sums' columns, its 64 groups of 16 lanes every 64th row each. A launch and two latencies: 4 us.
__global__ void __launch_bounds__(1024)
moe_rotary_reduce(const float* ws, float* out0, float* out1, int D, int sums, int rows) {
    __shared__ float part[64][17];
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4;
    const int col = blockIdx.x * 16 + lane;              // of sums * D
    float s = 0.0f;
    if (col < sums * D) {
#pragma unroll 16
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

// The runs of tokens of the backward kernel: as long as leave every compute unit one,
// with their turns in 32 KB of LDS.
int back_tokens(const mega_moe_rotary_backward_args& a) {
    const int most = a.rotary_dim > 0 ? 8192 / a.rotary_dim : 64;
    const int n = (a.num_tokens + BACK_BLOCKS - 1) / BACK_BLOCKS;
    return n < 1 ? 1 : n < most ? n : most;
}

// Its grid; few tokens: their heads over several workgroups.
dim3 back_grid(const mega_moe_rotary_backward_args& a) {
    const int tokens = back_tokens(a), need = (a.num_tokens + tokens - 1) / tokens;
    const int blocks = need < BACK_BLOCKS ? need : BACK_BLOCKS, G = BACK_THREADS / lanes_of(a.head_dim);
    const int rounds = (tokens * (a.q_heads + a.k_heads) + G - 1) / G, split = blocks > 0 ? BACK_BLOCKS / blocks : 1;
    return dim3((unsigned)blocks, (unsigned)(split < rounds ? split : rounds));
}

}  // namespace

namespace {

void launch_turned(const mega_moe_rotary_args& a, float sign, hipStream_t stream) {
    const int tokens = tokens_of(a.num_tokens, a.rotary_dim);
    const int blocks = (a.num_tokens + tokens - 1) / tokens;
    // few tokens: their heads over several workgroups
    const int G = THREADS / lanes_of(a.head_dim), rounds = (tokens * (a.q_heads + a.k_heads) + G - 1) / G;
    int split = (1024 + blocks - 1) / blocks;
    if (split > rounds) split = rounds;
    const unsigned lds = (unsigned)(tokens * a.rotary_dim * 4);
    const auto go = [&](auto f32) {
        by_lanes<decltype(f32)::value>(a, [&](auto lanes) {
            hipLaunchKernelGGL((moe_rotary<decltype(f32)::value, decltype(lanes)::value>), dim3((unsigned)blocks, (unsigned)split),
                               dim3(THREADS), lds, stream, a, tokens, sign);
        });
    };
    if (a.type == MEGA_MOE_F32) go(std::true_type());
    else go(std::false_type());
}

}  // namespace

void launch_rotary(const mega_moe_rotary_args& a, hipStream_t stream) { launch_turned(a, 1.0f, stream); }

int rotary_backward_blocks(const mega_moe_rotary_backward_args& a) {
    const dim3 g = back_grid(a);
    return (int)(g.x * g.y);
}

void launch_rotary_backward(const mega_moe_rotary_backward_args& a, hipStream_t stream) {
    if (!a.q_weight && !a.k_weight) {
        // gradients of the rotation alone: the rotation by the opposite angles (8192 tokens of 32 + 8 heads of
        // 128 in 36.8 us, in the kernel for weights 41.7)
        const mega_moe_rotary_args f = {a.num_tokens, a.q_heads, a.k_heads, a.head_dim, a.rotary_dim, a.rotary_start, a.layout, a.type,
                                        a.weight_type, a.first_position, a.eps, a.scale, a.dq_out, a.dk_out, nullptr, nullptr,
                                        a.positions, a.inv_freq, a.dq, a.dk, a.dq_out_stride, a.dk_out_stride, a.dq_stride,
                                        a.dk_stride, a.dq_out_head_stride, a.dk_out_head_stride, a.dq_head_stride, a.dk_head_stride};
        launch_turned(f, -1.0f, stream);
        return;
    }
    const int tokens = back_tokens(a), blocks = rotary_backward_blocks(a);
    const unsigned lds = (unsigned)(tokens * a.rotary_dim * 4);
    float* ws = static_cast<float*>(a.workspace);
    if (blocks > 0) {
        const auto go = [&](auto f32) {
            by_lanes<decltype(f32)::value>(a, [&](auto lanes) {
                hipLaunchKernelGGL((moe_rotary_backward<decltype(f32)::value, decltype(lanes)::value>), back_grid(a),
                                   dim3(BACK_THREADS), lds, stream, a, ws, tokens);
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
