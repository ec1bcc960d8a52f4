// The operands of the E4M3 products: rows of x, or of silu(x) * up, or of its
// gradients, as codes with scales, by rows, by columns and by blocks.
#include <hip/hip_runtime.h>

#include "block_util.h"
#include "quantize.h"

namespace mega_moe {

namespace {

// What the kernels compute of a row's eight columns.
constexpr int PLAIN = 0;        // h = x
constexpr int SWIGLU = 1;       // h = silu(x) * up
constexpr int GRAD = 2;         // dx and dup, of x, up and dh

// One argument block for all of them.
struct QuantArgs {
    const void* x;
    const void* up;
    const void* dh;
    void* out[2];               // h in BF16; dx and dup in x's type
    uint8_t* q;
    float* q_sf;
    uint8_t* qt;
    float* qt_sf;
    int64_t x_stride, up_stride, dh_stride, out_stride[2];
    int T, C;
    float clamp;                // infinite: none
};

// A block's scale and what its values are multiplied and divided by, from the
// largest magnitude as float32 bits (a NaN is the largest).
struct Scale {
    float sf, up, d, inv;
    __device__ explicit Scale(uint32_t m) {
        const float amax = __uint_as_float(m);
        sf = amax / 448.0f;
        // tiny blocks are scaled up first, so that the reciprocal is finite
        up = sf < 0x1p-100f ? 0x1p100f : 1.0f;
        d = (amax * up) / 448.0f;
        inv = amax == 0.0f ? 0.0f : 1.0f / d;
        if (inv == 0.0f) d = 0.0f;               // a scale of 0 or infinity: codes of 0
    }
    // v / sf, rounded as a division rounds it: the product with the reciprocal
    // and one step of Newton's iteration.
    __device__ __forceinline__ float quotient(float v) const {
        const float x = v * up, q = x * inv;
        return fmaf(-fmaf(q, d, -x), inv, q);
    }
    __device__ __forceinline__ uint32_t codes(float a, float b, float c, float e) const {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(a), quotient(b), 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(quotient(c), quotient(e), lo, true);
    }
};

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Of the smaller exponential, so that a low gate keeps its share down to the subnormals.
__device__ __forceinline__ float sigmoid(float g) {
    const float e = expf(-fabsf(g));
    return (g < 0.0f ? e : 1.0f) / (1.0f + e);
}

// The layer's clamp: fminf and fmaxf would turn a NaN into a bound.
__device__ __forceinline__ float clamped(float v, float c) { return v > c ? c : v < -c ? -c : v; }

// The eight values of output `which` from the raw inputs.
template <int KIND>
__device__ __forceinline__ void values(int which, float (&x)[8], const float (&up)[8], const float (&dh)[8], float clamp) {
    if constexpr (KIND == PLAIN) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float g = clamped(x[i], clamp), u = clamped(up[i], clamp);
        const float s = sigmoid(g);
        if constexpr (KIND == SWIGLU) {
            x[i] = g * s * u;
        } else {
            if (which == 0) x[i] = fabsf(x[i]) > clamp ? 0.0f : dh[i] * u * (s * (1.0f + g * (1.0f - s)));
            else x[i] = fabsf(up[i]) > clamp ? 0.0f : dh[i] * (g * s);
        }
    }
}

// Eight columns of one row as they lie in memory.
template <int KIND, bool F32>
struct Raw {
    static constexpr int N = F32 ? 2 : 1;
    u32x4_t x[N], up[N], dh[N];
    __device__ __forceinline__ void load(const QuantArgs& a, int64_t t, int col) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = raw8<F32>(a.x, t * a.x_stride + col)[i];
            if constexpr (KIND != PLAIN) up[i] = raw8<F32>(a.up, t * a.up_stride + col)[i];
            if constexpr (KIND == GRAD) dh[i] = raw8<F32>(a.dh, t * a.dh_stride + col)[i];
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = up[i] = dh[i] = u32x4_t{0u, 0u, 0u, 0u};
    }
    __device__ __forceinline__ void get(int which, float clamp, float (&v)[8]) const {
        float u[8] = {}, d[8] = {};
        values8<F32>(x, v);
        if constexpr (KIND != PLAIN) values8<F32>(up, u);
        if constexpr (KIND == GRAD) values8<F32>(dh, d);
        values<KIND>(which, v, u, d, clamp);
    }
};

template <int KIND, bool F32>
__device__ __forceinline__ void store_out(const QuantArgs& a, int which, int64_t t, int col, const float (&v)[8]) {
    if (!a.out[which]) return;
    if constexpr (KIND == GRAD) store8<F32>(a.out[which], t * a.out_stride[which] + col, v);
    else store8<false>(a.out[which], t * a.out_stride[which] + col, v);
}

}  // namespace

// Codes by rows and values alone: 16 lanes hold 128 columns of a row.
template <int KIND, bool F32>
__global__ void __launch_bounds__(256) moe_quantize_rows(QuantArgs a) {
    constexpr int OUTS = KIND == GRAD ? 2 : 1;
    const int blocks = a.C / 128, lane = threadIdx.x & 15;
    const int64_t items = (int64_t)a.T * blocks;
    for (int64_t i = (int64_t)blockIdx.x * 16 + threadIdx.x / 16; i < items; i += (int64_t)gridDim.x * 16) {
        const int64_t t = i / blocks;
        const int b = (int)(i - t * blocks), col = b * 128 + lane * 8;
        Raw<KIND, F32> raw;
        raw.load(a, t, col);
#pragma unroll
        for (int which = 0; which < OUTS; ++which) {
            float v[8];
            raw.get(which, a.clamp, v);
            store_out<KIND, F32>(a, which, t, col, v);
            if (!a.q) continue;
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = larger(m, magnitude(v[e]));
            m = over_lanes<16>(m, larger);
            const Scale s(m);
            const int64_t row = t * OUTS + which;        // [T, OUTS * C] codes
            *reinterpret_cast<uint2*>(a.q + row * a.C + col) =
                uint2{s.codes(v[0], v[1], v[2], v[3]), s.codes(v[4], v[5], v[6], v[7])};
            if (lane == 0) a.q_sf[row * blocks + b] = s.sf;
        }
    }
}

// Codes by columns, by blocks, and by rows beside them: a workgroup has a tile
// of 128 rows x 128 columns, a thread eight columns of four rows that follow
// each other.  A column's largest value is that of the thread's rows, of the
// wave's four groups of rows and, through LDS, of the eight waves.  The codes by
// columns turn in LDS: a thread has four neighbours of each, and a row of 128
// leaves as whole lines.
template <int KIND, bool F32, bool BLOCK>
__global__ void __launch_bounds__(512) moe_quantize_tile(QuantArgs a) {
    constexpr int OUTS = KIND == GRAD ? 2 : 1;
    __shared__ uint32_t top[8][128];
    __shared__ uint32_t turned[128 * 32];                // [column][4 rows], words swizzled
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int blocks = a.C / 128, row_blocks = (a.T + 127) / 128;
    const int64_t tiles = (int64_t)blocks * row_blocks;
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int rb = (int)(tile / blocks), b = (int)(tile - (int64_t)rb * blocks);
        const int col = b * 128 + lane * 8;
        const int64_t t0 = (int64_t)rb * 128 + group * 4;
        Raw<KIND, F32> raw[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            if (t0 + r < a.T) raw[r].load(a, t0 + r, col);
            else raw[r].zero();
        }
#pragma unroll
        for (int which = 0; which < OUTS; ++which) {
            float v[4][8];
            uint32_t m[4] = {};                          // by rows
            uint32_t mc[8] = {};                         // by columns
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                raw[r].get(which, a.clamp, v[r]);
                // rows behind the last are 0 whatever is made of zeros
                if (t0 + r < a.T) store_out<KIND, F32>(a, which, t0 + r, col, v[r]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t x = magnitude(v[r][e]);
                    m[r] = larger(m[r], x);
                    mc[e] = larger(mc[e], x);
                }
            }
            if constexpr (BLOCK) {
                uint32_t all = larger(larger(m[0], m[1]), larger(m[2], m[3]));
                all = over_lanes<64>(all, larger);
                if ((threadIdx.x & 63) == 0) top[wave][0] = all;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < 8; ++w) all = larger(all, top[w][0]);
                m[0] = all;
            } else {
                if (a.q) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) m[r] = over_lanes<16>(m[r], larger);
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    auto p = __builtin_amdgcn_permlane16_swap(mc[e], mc[e], false, false);
                    mc[e] = larger(p[0], p[1]);
                    p = __builtin_amdgcn_permlane32_swap(mc[e], mc[e], false, false);
                    mc[e] = larger(p[0], p[1]);
                }
                if ((threadIdx.x & 63) < 16) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) top[wave][lane * 8 + e] = mc[e];
                }
                __syncthreads();
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int w = 0; w < 8; ++w) mc[e] = larger(mc[e], top[w][lane * 8 + e]);
            }
            if (a.q) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const Scale s(m[BLOCK ? 0 : r]);
                    if (t0 + r >= a.T) continue;
                    const int64_t row = (t0 + r) * OUTS + which;
                    *reinterpret_cast<uint2*>(a.q + row * a.C + col) =
                        uint2{s.codes(v[r][0], v[r][1], v[r][2], v[r][3]), s.codes(v[r][4], v[r][5], v[r][6], v[r][7])};
                    if (!BLOCK && lane == 0) a.q_sf[row * blocks + b] = s.sf;
                    if (BLOCK && threadIdx.x == 0 && r == 0) a.q_sf[(int64_t)rb * blocks + b] = s.sf;
                }
            }
            if (a.qt) {
                const int64_t row0 = (int64_t)which * a.C + b * 128;     // of qt
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const Scale s(BLOCK ? m[0] : mc[e]);
                    // the eight threads' words of four that a row's 16 bytes are spread over the banks
                    turned[(lane * 8 + e) * 32 + (group ^ ((lane & 7) * 4))] = s.codes(v[0][e], v[1][e], v[2][e], v[3][e]);
                    if (!BLOCK && group == 0) a.qt_sf[(row0 + lane * 8 + e) * row_blocks + rb] = s.sf;
                    if (BLOCK && threadIdx.x == 0 && e == 0) a.qt_sf[(int64_t)b * row_blocks + rb] = s.sf;
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int c = (threadIdx.x >> 3) + 64 * i, w = (threadIdx.x & 7) * 4;
                    const u32x4_t d = *reinterpret_cast<const u32x4_t*>(&turned[c * 32 + (w ^ (((c >> 3) & 7) * 4))]);
                    *reinterpret_cast<u32x4_t*>(a.qt + (row0 + c) * ((int64_t)row_blocks * 128) + (int64_t)rb * 128 + w * 4) = d;
                }
            }
            __syncthreads();                             // top and turned are written again
        }
    }
}

namespace {

// Workgroups at most: the kernels go on to the next item behind them.
constexpr int64_t MAX_GRID = 1 << 20;

template <int KIND, bool F32>
void launch(const QuantArgs& a, bool block, hipStream_t stream) {
    if (a.qt || (block && a.q)) {
        const int64_t tiles = (int64_t)(a.C / 128) * ((a.T + 127) / 128);
        const auto go = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles < MAX_GRID ? tiles : MAX_GRID)), dim3(512), 0, stream, a);
        };
        if (KIND != GRAD && block) go(moe_quantize_tile<KIND, F32, KIND != GRAD>);
        else go(moe_quantize_tile<KIND, F32, false>);
    } else {
        const int64_t n = ((int64_t)a.T * (a.C / 128) + 15) / 16;
        hipLaunchKernelGGL((moe_quantize_rows<KIND, F32>), dim3((unsigned)(n < MAX_GRID ? n : MAX_GRID)), dim3(256), 0, stream, a);
    }
}

}  // namespace

void launch_quantize(const mega_moe_quantize_args& g, hipStream_t stream) {
    const QuantArgs a = {g.x, g.up, nullptr, {g.h, nullptr}, g.q, g.q_sf, g.qt, g.qt_sf, g.x_stride, g.up_stride, 0,
                         {g.h_stride, 0}, g.num_tokens, g.columns, g.activation_clamp == 0.0f ? INFINITY : g.activation_clamp};
    const bool f = g.x_type == MEGA_MOE_F32, block = g.scale == MEGA_MOE_SCALE_BLOCK;
    if (g.activation == MEGA_MOE_ACT_SWIGLU) f ? launch<SWIGLU, true>(a, block, stream) : launch<SWIGLU, false>(a, block, stream);
    else f ? launch<PLAIN, true>(a, block, stream) : launch<PLAIN, false>(a, block, stream);
}

void launch_swiglu_backward(const mega_moe_swiglu_backward_args& g, hipStream_t stream) {
    const QuantArgs a = {g.x, g.up, g.dh, {g.dx, g.dup}, g.q, g.q_sf, g.qt, g.qt_sf, g.x_stride, g.up_stride, g.dh_stride,
                         {g.dx_stride, g.dup_stride}, g.num_tokens, g.columns,
                         g.activation_clamp == 0.0f ? INFINITY : g.activation_clamp};
    if (g.x_type == MEGA_MOE_F32) launch<GRAD, true>(a, false, stream);
    else launch<GRAD, false>(a, false, stream);
}

}  // namespace mega_moe
