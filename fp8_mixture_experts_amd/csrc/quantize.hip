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

// As the layer clamps: fminf and fmaxf would turn a NaN into a bound.
__device__ __forceinline__ float clamped(float v, float c) { return v > c ? c : v < -c ? -c : v; }

// A block's scale, and what its values are multiplied by, from the largest magnitude
// as float32 bits (a NaN is the largest).
struct Scale {
    float sf, up, hi, lo;        // sf = 1 / ((hi + lo) up), to 2^-46
    Scale() = default;
    __device__ __forceinline__ explicit Scale(uint32_t m) {
        const float amax = __uint_as_float(m);
        sf = amax / 448.0f;
        // tiny blocks are scaled up first, so that the reciprocal is finite, and large ones down, so
        // that what is left of it is no subnormal number (from scales of 2^102 on it would lose bits)
        up = sf < 0x1p-100f ? 0x1p100f : sf > 0x1p64f ? 0x1p-64f : 1.0f;
        const float d = sf * up;             // exact, also of a subnormal scale
        hi = d == 0.0f ? 0.0f : 1.0f / d;
        // a scale of 0 or infinity: codes of 0
        lo = hi == 0.0f ? 0.0f : fmaf(-d, hi, 1.0f) * hi;
    }
    // That of lane L of the lane's four.
    template <int L>
    __device__ __forceinline__ Scale of_quad() const {
        const auto move = [](float v) {
            return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x55 * L, 0xf, 0xf, true));
        };
        Scale o;
        o.sf = 0.0f;
        o.up = move(up), o.hi = move(hi), o.lo = move(lo);
        return o;
    }
    // v / sf: one rounding of a sum that is off by 2^-46, so that it is the quotient's own
    // but within that of the middle between two floats; no tie between codes lies there.
    // (A subnormal scale may be rounded down by up to a third: the largest code then.)
    template <bool SCALED>
    __device__ __forceinline__ float quotient(float v) const {
        if constexpr (SCALED) v *= up;
        const float q = fmaf(v, hi, v * lo);
        return SCALED ? clamped(q, 448.0f) : q;
    }
    template <bool SCALED>
    __device__ __forceinline__ uint32_t codes(float a, float b, float c, float e) const {
        const int p = __builtin_amdgcn_cvt_pk_fp8_f32(quotient<SCALED>(a), quotient<SCALED>(b), 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(quotient<SCALED>(c), quotient<SCALED>(e), p, true);
    }
};

// The larger magnitude; of a NaN and another, the NaN.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(fabsf(a), fabsf(b)); }
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// s = 1 / (1 + exp(-g)), of the smaller exponential, so that a low gate keeps its share
// down to the subnormals.  exp(-|g|) is the square of 2^(-|g| log2(e) / 2), whose
// argument's rounding error (and log2(e)'s) is put back to first order: the square root is a normal number
// wherever the square is not 0. 1 + e is in [1, 2], where the hardware's reciprocal and one
// step of Newton's iteration leave an error below a step.
__device__ __forceinline__ float sigmoid(float g) {
    constexpr float HALF_LOG2E = 0.72134751081466675f, REST = 9.6298151675e-9f, TWO_LN2 = 1.3862943611198906f;
    const float a = -fminf(fabsf(g), 256.0f), x = a * HALF_LOG2E;
    const float off = fmaf(a, REST, fmaf(a, HALF_LOG2E, -x)), h = __builtin_amdgcn_exp2f(x), hh = h * h;
    const float e = fmaf(hh, off * TWO_LN2, hh), t = 1.0f + e, r = __builtin_amdgcn_rcpf(t);
    return (g < 0.0f ? e : 1.0f) * fmaf(fmaf(-t, r, 1.0f), r, r);
}

// Eight columns of one row as they lie in memory, and what is made of them.
template <int KIND, bool F32>
struct Raw {
    static constexpr int N = F32 ? 2 : 1, OUTS = KIND == GRAD ? 2 : 1;
    u32x4_t x[N], up[N], dh[N];
    // (zeros where the row is none)
    __device__ __forceinline__ void load(const QuantArgs& a, int64_t t, int col, bool live) {
        const u32x4_t none = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < N; ++i) {
            x[i] = live ? raw8<F32>(a.x, t * a.x_stride + col)[i] : none;
            if constexpr (KIND != PLAIN) up[i] = live ? raw8<F32>(a.up, t * a.up_stride + col)[i] : none;
            if constexpr (KIND == GRAD) dh[i] = live ? raw8<F32>(a.dh, t * a.dh_stride + col)[i] : none;
        }
    }
    // (the clamp is uniform, and mostly there is none)
    __device__ __forceinline__ void get(float clamp, float (&v)[OUTS][8]) const {
        if (KIND == PLAIN || clamp == INFINITY) make<false>(clamp, v);
        else make<true>(clamp, v);
    }
    template <bool CLAMP>
    __device__ __forceinline__ void make(float clamp, float (&v)[OUTS][8]) const {
        float g[8], u[8] = {}, d[8] = {};
        values8<F32>(x, g);
        if constexpr (KIND != PLAIN) values8<F32>(up, u);
        if constexpr (KIND == GRAD) values8<F32>(dh, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (KIND == PLAIN) {
                v[0][i] = g[i];
            } else {
                const float gc = CLAMP ? clamped(g[i], clamp) : g[i], uc = CLAMP ? clamped(u[i], clamp) : u[i], s = sigmoid(gc);
                if constexpr (KIND == SWIGLU) {
                    v[0][i] = gc * s * uc;
                } else {
                    v[0][i] = CLAMP && fabsf(g[i]) > clamp ? 0.0f : d[i] * uc * (s * (1.0f + gc * (1.0f - s)));
                    v[OUTS - 1][i] = CLAMP && fabsf(u[i]) > clamp ? 0.0f : d[i] * (gc * s);
                }
            }
        }
    }
};

template <int KIND, bool F32>
__device__ __forceinline__ void store_out(const QuantArgs& a, int which, int64_t t, int col, const float (&v)[8]) {
    if (!a.out[which]) return;
    if constexpr (KIND == GRAD) store8<F32>(a.out[which], t * a.out_stride[which] + col, v);
    else store8<false>(a.out[which], t * a.out_stride[which] + col, v);
}

}  // namespace

// Codes by rows and values alone: 16 lanes hold 128 columns of a row, whose largest value they find in four
// lane moves.  One pass over the data: the launch bounds small batches (128 x 2048 of SwiGLU 7.1 us with the
// call, 3.0 the kernel; 577 x 2048 gradients 6.7), memory large ones.
template <int KIND, bool F32>
__global__ void __launch_bounds__(256) moe_quantize_rows(QuantArgs a) {
    constexpr int OUTS = KIND == GRAD ? 2 : 1;
    const int blocks = a.C / 128, lane = threadIdx.x & 15;
    const int64_t items = (int64_t)a.T * blocks;
    for (int64_t i = (int64_t)blockIdx.x * 16 + threadIdx.x / 16; i < items; i += (int64_t)gridDim.x * 16) {
        const int64_t t = i / blocks;
        const int b = (int)(i - t * blocks), col = b * 128 + lane * 8;
        Raw<KIND, F32> raw;
        raw.load(a, t, col, true);
        float made[OUTS][8];
        raw.get(a.clamp, made);
#pragma unroll
        for (int which = 0; which < OUTS; ++which) {
            const float (&v)[8] = made[which];
            store_out<KIND, F32>(a, which, t, col, v);
            if (!a.q) continue;
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = larger(m, v[e]);
            const Scale s(over_lanes<16>(__float_as_uint(m), [](uint32_t x, uint32_t y) { return larger(x, y); }));
            const int64_t row = t * OUTS + which;        // [T, OUTS * C] codes
            const auto row_codes = [&](auto scaled) {
                constexpr bool SCALED = decltype(scaled)::value;
                *reinterpret_cast<uint2*>(a.q + row * a.C + col) =
                    uint2{s.codes<SCALED>(v[0], v[1], v[2], v[3]), s.codes<SCALED>(v[4], v[5], v[6], v[7])};
            };
            if (__any(s.up != 1.0f)) row_codes(std::true_type());
            else row_codes(std::false_type());
            if (lane == 0) a.q_sf[row * blocks + b] = s.sf;
        }
    }
}

// The largest of eight columns over the wave's four groups of 16 lanes: the columns
// part as the groups meet, so that a lane is left with two of its eight, from columns_of() on.
__device__ __forceinline__ uint2 over_groups(const uint32_t (&m)[8]) {
    uint32_t four[4], two[2];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const auto p = __builtin_amdgcn_permlane16_swap(m[e], m[e + 4], false, false);
        four[e] = larger(p[0], p[1]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        const auto p = __builtin_amdgcn_permlane32_swap(four[e], four[e + 2], false, false);
        two[e] = larger(p[0], p[1]);
    }
    return uint2{two[0], two[1]};
}
__device__ __forceinline__ int columns_of() { return (threadIdx.x & 16) / 4 + (threadIdx.x & 32) / 16; }

// Codes by columns, by blocks, and by rows beside them: a workgroup has a tile
// of 128 rows x 128 columns, a thread eight columns of R rows that follow
// each other.  A column's largest value is that of the thread's rows, of the
// wave's four groups of rows and, through LDS, of the waves; its scale is worked
// out by one thread, a row's by one of the row's lanes (three divisions each, of
// which a thread would have 36).  The codes by columns turn in LDS: a thread has R
// neighbours of each, and a row of 128 leaves as whole lines.
//
// One pass: 8192 x 7168 BF16 to codes by rows and by columns 54 us (239 MB, 4.4 TB/s with the call; a copy's rate
// would be 47), SwiGLU gradients 4096 x 2048 to both 20.3 us (85 MB; 16.7): vector instructions have 40% and
// 44% of the cycles, beside the memory, and a compute unit's tiles start and end together.
//
// Four waves to a vector unit (two workgroups of 8 to a compute unit, or one of 16): the gradients' codes fill
// the registers that this leaves, and with two more take 26.7 us, not 20.5.
template <int KIND, bool F32, bool BLOCK, int R>
__global__ void __launch_bounds__(2048 / R, 4) moe_quantize_tile(QuantArgs a) {
    constexpr int OUTS = KIND == GRAD ? 2 : 1, WAVES = 32 / R;
    constexpr bool AHEAD = R == 2 && !F32;               // the next tile's loads in flight behind this one's codes
    __shared__ __attribute__((aligned(16))) uint32_t top[OUTS][WAVES][128];
    __shared__ __attribute__((aligned(16))) float col_up[OUTS * 128], col_hi[OUTS * 128], col_lo[OUTS * 128];
    __shared__ int col_scaled[OUTS * 2];
    __shared__ __attribute__((aligned(16))) uint8_t turned[OUTS][128 * 128];   // [column][row], chunks of 16 swizzled
    const int lane = threadIdx.x & 15, group = threadIdx.x >> 4, wave = threadIdx.x >> 6;
    const int blocks = a.C / 128, row_blocks = (a.T + 127) / 128;
    const int64_t tiles = (int64_t)blocks * row_blocks;
    typedef Raw<KIND, F32> Rows[R];
    const auto fetch = [&](Rows& raw, int64_t tile) {
        const int64_t rb = tile / blocks, t = rb * 128 + group * R;
        const int col = (int)(tile - rb * blocks) * 128 + lane * 8;
#pragma unroll
        for (int r = 0; r < R; ++r) raw[r].load(a, t + r, col, t + r < a.T);
    };
    const auto max_bits = [](uint32_t x, uint32_t y) { return larger(x, y); };
    Rows ahead;
    if constexpr (AHEAD) {
        if (blockIdx.x < tiles) fetch(ahead, blockIdx.x);
    }
    for (int64_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
        const int rb = (int)(tile / blocks), b = (int)(tile - (int64_t)rb * blocks);
        const int col = b * 128 + lane * 8;
        const int64_t t0 = (int64_t)rb * 128 + group * R;
        const auto qt_row = [&](int c) { return (int64_t)(c / 128) * a.C + b * 128 + (c & 127); };
        Rows here;
        if constexpr (!AHEAD) fetch(here, tile);
        float made[OUTS][R][8];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float v[OUTS][8];
            if constexpr (AHEAD) ahead[r].get(a.clamp, v);
            else here[r].get(a.clamp, v);
#pragma unroll
            for (int which = 0; which < OUTS; ++which) {
                // rows behind the last are 0 whatever is made of zeros
                if (t0 + r < a.T) store_out<KIND, F32>(a, which, t0 + r, col, v[which]);
#pragma unroll
                for (int e = 0; e < 8; ++e) made[which][r][e] = v[which][e];
            }
        }
        if constexpr (AHEAD) {
            if (tile + gridDim.x < tiles) fetch(ahead, tile + gridDim.x);
        }
        uint32_t most[OUTS][R];                          // of the thread's part of a row
        Scale of_block;
#pragma unroll
        for (int which = 0; which < OUTS; ++which) {
            const float (&v)[R][8] = made[which];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                float m = larger(v[r][0], v[r][1]);
#pragma unroll
                for (int e = 2; e < 8; e += 2) m = larger(larger(v[r][e], v[r][e + 1]), m);
                most[which][r] = __float_as_uint(m);
            }
            if constexpr (BLOCK) {
                uint32_t all = most[which][0];
#pragma unroll
                for (int r = 1; r < R; ++r) all = larger(all, most[which][r]);
                all = over_lanes<64>(all, max_bits);
                if ((threadIdx.x & 63) == 0) top[which][wave][0] = all;
            } else {
                uint32_t bits[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float m = larger(v[0][e], v[1][e]);
#pragma unroll
                    for (int r = 2; r < R; r += 2) m = larger(larger(v[r][e], v[r + 1][e]), m);
                    bits[e] = __float_as_uint(m);
                }
                *reinterpret_cast<uint2*>(&top[which][wave][lane * 8 + columns_of()]) = over_groups(bits);
            }
        }
        __syncthreads();
        if constexpr (BLOCK) {
            uint32_t all = top[0][0][0];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) all = larger(all, top[0][w][0]);
            of_block = Scale(all);
            if (threadIdx.x == 0) {
                if (a.q) a.q_sf[(int64_t)rb * blocks + b] = of_block.sf;
                if (a.qt) a.qt_sf[(int64_t)b * row_blocks + rb] = of_block.sf;
            }
        } else if (threadIdx.x < OUTS * 128) {
            const int which = OUTS == 1 ? 0 : threadIdx.x >> 7, c = threadIdx.x & 127;
            uint32_t x = top[which][0][c];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) x = larger(x, top[which][w][c]);
            const Scale s(x);
            a.qt_sf[qt_row(threadIdx.x) * row_blocks + rb] = s.sf;
            col_up[threadIdx.x] = s.up, col_hi[threadIdx.x] = s.hi, col_lo[threadIdx.x] = s.lo;
            const bool scaled = __any(s.up != 1.0f);
            if ((threadIdx.x & 63) == 0) col_scaled[wave] = scaled;
        }
        if (a.q) {
#pragma unroll
            for (int which = 0; which < OUTS; ++which) {
                const float (&v)[R][8] = made[which];
                Scale mine = of_block;
                if constexpr (!BLOCK) {
                    uint32_t bits[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) bits[r] = over_lanes<16>(most[which][r], max_bits);
                    uint32_t own = lane & 1 ? bits[1] : bits[0];
                    if constexpr (R == 4) own = lane & 2 ? (lane & 1 ? bits[3] : bits[2]) : own;
                    mine = Scale(own);
                    if (lane < R && t0 + lane < a.T) a.q_sf[((t0 + lane) * OUTS + which) * blocks + b] = mine.sf;
                }
                const auto row_codes = [&](auto scaled) {
                    constexpr bool SCALED = decltype(scaled)::value;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const Scale s = r == 0 ? mine.of_quad<0>() : r == 1 ? mine.of_quad<1>() : r == 2 ? mine.of_quad<2>() : mine.of_quad<3>();
                        const uint2 d = {s.codes<SCALED>(v[r][0], v[r][1], v[r][2], v[r][3]), s.codes<SCALED>(v[r][4], v[r][5], v[r][6], v[r][7])};
                        if (t0 + r < a.T) *reinterpret_cast<uint2*>(a.q + ((t0 + r) * OUTS + which) * a.C + col) = d;
                    }
                };
                if (__any(mine.up != 1.0f)) row_codes(std::true_type());
                else row_codes(std::false_type());
            }
        }
        if (a.qt) {
            if (!BLOCK) __syncthreads();
#pragma unroll
            for (int which = 0; which < OUTS; ++which) {
                const float (&v)[R][8] = made[which];
                const auto column_codes = [&](auto scaled) {
                    constexpr bool SCALED = decltype(scaled)::value;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        Scale s = of_block;
                        if constexpr (!BLOCK) {
                            const int c = which * 128 + lane * 8 + e;
                            s.hi = col_hi[c], s.lo = col_lo[c];
                            if constexpr (SCALED) s.up = col_up[c];
                        }
                        // the 16 bytes of a row lie at chunk ^ (column / 8 % 8)
                        uint8_t* to = turned[which] + (lane * 8 + e) * 128 + ((group * R) ^ ((lane & 7) * 16));
                        if constexpr (R == 4) *reinterpret_cast<uint32_t*>(to) = s.codes<SCALED>(v[0][e], v[1][e], v[2][e], v[R - 1][e]);
                        else *reinterpret_cast<uint16_t*>(to) = (uint16_t)__builtin_amdgcn_cvt_pk_fp8_f32(s.quotient<SCALED>(v[0][e]), s.quotient<SCALED>(v[1][e]), 0, false);
                    }
                };
                if (BLOCK ? of_block.up != 1.0f : (col_scaled[2 * which] | col_scaled[2 * which + 1]) != 0) column_codes(std::true_type());
                else column_codes(std::false_type());
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < OUTS * R / 2; ++i) {
                const int c = (threadIdx.x >> 3) + 256 / R * i, w = (threadIdx.x & 7) * 16;
                const u32x4_t d = *reinterpret_cast<const u32x4_t*>(turned[0] + c * 128 + (w ^ (((c >> 3) & 7) * 16)));
                *reinterpret_cast<u32x4_t*>(a.qt + qt_row(c) * ((int64_t)row_blocks * 128) + (int64_t)rb * 128 + w) = d;
            }
        }
        if (BLOCK) __syncthreads();                      // top is written again (else two barriers lie between)
    }
}

namespace {

// Workgroups at most: the kernels go on to the next item behind them.
constexpr int64_t MAX_GRID = 1 << 20;

template <int KIND, bool F32>
void launch(const QuantArgs& a, bool block, hipStream_t stream) {
    if (a.qt || (block && a.q)) {
        const int64_t tiles = (int64_t)(a.C / 128) * ((a.T + 127) / 128);
        const auto go = [&](auto kernel, int rows, int64_t most) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)(tiles < most ? tiles : most)), dim3(2048 / rows), 0, stream, a);
        };
        if constexpr (KIND == GRAD) {
            // The values of two outputs leave a compute unit two workgroups of 8 waves with four rows to a
            // thread, or one of 16 with two, which goes on to further tiles, with their loads in flight
            // (float32's do not fit beside the values; with four rows float32 has scratch).  Codes of BF16 alone are
            // better made by the former, with the gradients stored too and of float32 by the latter.  Both ways, us
            // (four rows, two):
            //                      1000 x 4096   4096 x 2048   8192 x 2048   2304 x 7168   8192 x 4096
            //   codes              13.9  13.1    20.0  21.8    44.0  45.2    42.4  45.0    79.5   81.5
            //   codes, gradients   14.8  14.2    34.9  28.5    59.6  57.2    57.2  56.3    107.1  108.4
            //   float32, codes     19.4  15.0    41.1  36.2    75.5  66.2    73.8  66.8
            // and within 4% of each other below 256 tiles (float32 two rows: 15%).
            if (F32 || a.out[0] || a.out[1]) go(moe_quantize_tile<KIND, F32, false, 2>, 2, 256);
            else go(moe_quantize_tile<KIND, false, false, 4>, 4, MAX_GRID);
        } else if (block) {
            go(moe_quantize_tile<KIND, F32, true, 4>, 4, MAX_GRID);
        } else {
            go(moe_quantize_tile<KIND, F32, false, 4>, 4, MAX_GRID);
        }
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
