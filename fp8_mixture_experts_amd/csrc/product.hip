// out = a . b^T + add of E4M3 codes with float scales for 128 columns: of a's
// rows, and of b's rows or 128 x 128 blocks.
#include <hip/hip_runtime.h>

#include "block_util.h"
#include "product.h"

namespace mega_moe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));

constexpr int BK = 128;              // columns of a step: one scale block

struct ProductArgs {
    const uint8_t* a;
    const uint8_t* b;
    const float* a_sf;
    const float* b_sf;
    const void* add;
    void* out;
    float* parts;                    // [splits][m][n] with more than one split
    int64_t a_stride, b_stride, a_sf_stride, b_sf_stride, add_stride, out_stride;
    int m, n, steps, splits;
};

// A buffer over `bytes` bytes at `base` (both the same for the wave): loads
// beyond it give 0.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, uint32_t bytes) {
    const uint64_t p = (uint64_t)(uintptr_t)base;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
    return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)((uint64_t)hi << 32 | lo), 0,
                                             (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}

// 16 bytes a lane straight into LDS: lane L writes lds + 16 L.
__device__ __forceinline__ void load16_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, int voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, soff, 0, 0);
}

// 4 bytes a lane: lane L writes lds + 4 L.
__device__ __forceinline__ void load4_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, int voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 4, voff, soff, 0, 0);
}

// A stage's rows are 128 bytes; their 16-byte chunk c lies at c ^ turn(row), so
// that a load instruction covers eight whole rows and the 32 rows of a matrix
// operand meet distinct banks.
__device__ __forceinline__ int turn(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// The operand of 32 rows (slice s) for half h of a step: lane r + 32 g has row
// r, chunks 4 h + g and 4 h + 2 + g (alike for a and b).  Every read of a stage is one
// of integers: of other types the compiler would wait for all loads into LDS first.
__device__ __forceinline__ i32x8_t operand(const uint8_t* rows, int s, int h) {
    const int r = threadIdx.x & 31, g = (threadIdx.x >> 5) & 1;
    const uint8_t* row = rows + (32 * s + r) * BK;
    const i32x4_t lo = *reinterpret_cast<const i32x4_t*>(row + 16 * ((4 * h + g) ^ turn(r)));
    const i32x4_t hi = *reinterpret_cast<const i32x4_t*>(row + 16 * ((4 * h + 2 + g) ^ turn(r)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// A quarter (16 bytes a lane: 32 columns) of the same, for the F16 products.
__device__ __forceinline__ i32x4_t quarter(const uint8_t* rows, int s, int p) {
    const int r = threadIdx.x & 31, g = (threadIdx.x >> 5) & 1;
    return *reinterpret_cast<const i32x4_t*>(rows + (32 * s + r) * BK + 16 * ((2 * p + g) ^ turn(r)));
}

// Eight codes as F16: exact.
__device__ __forceinline__ f16x8_t half_values(int lo, int hi) {
    const f16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const f16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const f16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const f16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return f16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ f32x16_t product_f8(const i32x8_t& a, const i32x8_t& b, const f32x16_t& c) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);   // scales 0: none
}

// Tiles.  BM x BN results, by WM x WN waves, S steps in LDS.
template <int BM_, int BN_, int WM_, int WN_, int S_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, S = S_;
    static constexpr int NW = WM * WN, NT = 64 * NW;
    static constexpr int TM = BM / WM, TN = BN / WN;       // a wave's
    static constexpr int SM = TM / 32, SN = TN / 32;
    static constexpr int A_LOADS = BM / 8 / NW, B_LOADS = BN / 8 / NW;     // of 1 KB
    static constexpr int A_SF = BM / NW, B_SF = BN / NW;   // scales that a wave loads, a lane each
    static constexpr int OFF_B = BM * BK, OFF_SFA = OFF_B + BN * BK, OFF_SFB = OFF_SFA + BM * 4;
    template <bool ROWS>
    static constexpr int stage() { return OFF_SFB + (ROWS ? BN * 4 : 0); }
    template <bool ROWS>
    static constexpr int loads() { return A_LOADS + B_LOADS + 1 + (ROWS ? 1 : 0); }
    // results leave through LDS, PW columns of a wave at a time
    static constexpr int PW = TN < 64 ? TN : 64, PITCH = PW + 4;
    template <bool ROWS>
    static constexpr int lds() {
        const int a = S * stage<ROWS>(), b = NW * TM * PITCH * 4;
        return a > b ? a : b;
    }
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0 && A_SF <= 64 && B_SF <= 64, "loads");
};

// What workgroup `id` of `total` computes: the runs of ids that go to one of the
// eight dies (id % 8) are neighbours in the order.
__device__ __forceinline__ int in_order(int id, int total) {
    const int die = id & 7, q = total >> 3, r = total & 7;
    return die * q + (die < r ? die : r) + (id >> 3);
}

}  // namespace

// One tile, or one of `splits` parts of its steps.  b's rows are the matrix
// instruction's first operand, a's the second, so that a lane has one row of
// the result (32 of a slice) and register v column 8 (v / 4) + 4 (lane / 32) + v % 4: the
// scale of a's row is one value for a lane.
template <typename T, bool EXACT, bool ROWS>
__global__ void __launch_bounds__(T::NT) moe_product(ProductArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int STAGE = T::template stage<ROWS>(), LOADS = T::template loads<ROWS>(), S = T::S;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = w / T::WN, wn = w % T::WN;
    const int tiles_m = (p.m + T::BM - 1) / T::BM, tiles_n = (p.n + T::BN - 1) / T::BN;
    int at = in_order(blockIdx.x, gridDim.x);
    const int split = at / (tiles_m * tiles_n);
    at -= split * tiles_m * tiles_n;
    // eight rows of tiles at a time: neighbours share their rows of a and of b
    const int band = at / (8 * tiles_n), rows_of_band = min(8, tiles_m - band * 8);
    at -= band * 8 * tiles_n;
    const int64_t m0 = (int64_t)(band * 8 + at % rows_of_band) * T::BM, n0 = (int64_t)(at / rows_of_band) * T::BN;
    const int step0 = (int)((int64_t)p.steps * split / p.splits);
    const int steps = (int)((int64_t)p.steps * (split + 1) / p.splits) - step0;

    const int rows_a = (int)min((int64_t)T::BM, p.m - m0), rows_b = (int)min((int64_t)T::BN, p.n - n0);
    const __amdgpu_buffer_rsrc_t ra = buffer(p.a + m0 * p.a_stride + (int64_t)step0 * BK,
                                             (uint32_t)((rows_a - 1) * p.a_stride + (int64_t)steps * BK));
    const __amdgpu_buffer_rsrc_t rb = buffer(p.b + n0 * p.b_stride + (int64_t)step0 * BK,
                                             (uint32_t)((rows_b - 1) * p.b_stride + (int64_t)steps * BK));
    const __amdgpu_buffer_rsrc_t rsa = buffer(p.a_sf + m0 * p.a_sf_stride + step0,
                                              (uint32_t)((rows_a - 1) * p.a_sf_stride + steps) * 4);
    const __amdgpu_buffer_rsrc_t rsb = buffer(ROWS ? p.b_sf + n0 * p.b_sf_stride + step0 : nullptr,
                                              ROWS ? (uint32_t)((rows_b - 1) * p.b_sf_stride + steps) * 4 : 0u);
    // a wave's rows of a step: 8 (NW j + w) + lane / 8, and the chunk that belongs to lane % 8;
    // rows behind the last lie beyond the buffer by this offset alone
    const int r8 = 8 * w + (lane >> 3);
    const int voff_a = r8 * (int)p.a_stride + 16 * ((lane & 7) ^ turn(r8));
    const int voff_b = r8 * (int)p.b_stride + 16 * ((lane & 7) ^ turn(r8));
    static_assert((8 * T::NW) % 16 == 0 || T::NW == 1, "turn() is the same for a wave's rows");
    const int jump_a = 8 * T::NW * (int)p.a_stride, jump_b = 8 * T::NW * (int)p.b_stride;
    const int voff_sfa = (w * T::A_SF + min(lane, T::A_SF - 1)) * (int)p.a_sf_stride * 4;
    const int voff_sfb = (w * T::B_SF + min(lane, T::B_SF - 1)) * (int)p.b_sf_stride * 4;

    // The same number of instructions for every step, past the last one too.
    const auto issue = [&](int i) {
        uint8_t* stage = lds + (i % S) * STAGE;
        const bool real = i < steps;
        const int k = real ? i : 0;
        if (real || lane == 0) {
#pragma unroll
            for (int j = 0; j < T::A_LOADS; ++j)
                load16_lds(ra, stage + (T::NW * j + w) * 1024, voff_a + j * jump_a, k * BK);
#pragma unroll
            for (int j = 0; j < T::B_LOADS; ++j)
                load16_lds(rb, stage + T::OFF_B + (T::NW * j + w) * 1024, voff_b + j * jump_b, k * BK);
        }
        if (lane < T::A_SF && (real || lane == 0)) load4_lds(rsa, stage + T::OFF_SFA + w * T::A_SF * 4, voff_sfa, k * 4);
        if constexpr (ROWS) {
            if (lane < T::B_SF && (real || lane == 0)) load4_lds(rsb, stage + T::OFF_SFB + w * T::B_SF * 4, voff_sfb, k * 4);
        }
    };

    // b's block of scales: one for the wave (tiles start and end with blocks, or within one)
    const int64_t last_block = (p.n - 1) / 128;
    const float* b_sf = ROWS ? nullptr : p.b_sf + min((n0 + wn * T::TN) / 128, last_block) * p.b_sf_stride + step0;
    static_assert(T::TN == 128 || 128 % T::TN == 0, "one block of scales to a wave");

    f32x16_t acc[T::SN][T::SM];
#pragma unroll
    for (int j = 0; j < T::SN; ++j)
#pragma unroll
        for (int i = 0; i < T::SM; ++i) acc[j][i] = f32x16_t{};

    const auto add_step = [&](const uint8_t* stage, int step, const f32x16_t& d, int j, int i, float sa) {
        if constexpr (ROWS) {
            const uint8_t* sfb = stage + T::OFF_SFB + (wn * T::TN + 32 * j + ((lane >> 5) & 1) * 4) * 4;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const i32x4_t s = *reinterpret_cast<const i32x4_t*>(sfb + q * 32);
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[j][i][4 * q + e] = fmaf(d[4 * q + e], sa * __int_as_float(s[e]), acc[j][i][4 * q + e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[j][i][e] = fmaf(d[e], sa, acc[j][i][e]);
        }
    };

    if (steps > 0) {
#pragma unroll
        for (int i = 0; i < S - 1; ++i) issue(i);
        for (int step = 0; step < steps; ++step) {
            // this wave's loads of the step are there, then every wave's
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * LOADS) : "memory");
            issue(step + S - 1);
            const uint8_t* stage = lds + (step % S) * STAGE;
            const uint8_t* rows_x = stage + wm * T::TM * BK;
            const uint8_t* rows_w = stage + T::OFF_B + wn * T::TN * BK;
            const float sb = ROWS ? 1.0f : b_sf[step];
            float sa[T::SM];
#pragma unroll
            for (int i = 0; i < T::SM; ++i)
                sa[i] = sb * __int_as_float(*reinterpret_cast<const int*>(stage + T::OFF_SFA + (wm * T::TM + 32 * i + (lane & 31)) * 4));
            if constexpr (EXACT) {
                f32x16_t d[T::SN][T::SM];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    i32x4_t x[T::SM], y[T::SN];
#pragma unroll
                    for (int i = 0; i < T::SM; ++i) x[i] = quarter(rows_x, i, q);
#pragma unroll
                    for (int j = 0; j < T::SN; ++j) y[j] = quarter(rows_w, j, q);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f16x8_t xh[T::SM];
#pragma unroll
                        for (int i = 0; i < T::SM; ++i) xh[i] = half_values(x[i][2 * h], x[i][2 * h + 1]);
#pragma unroll
                        for (int j = 0; j < T::SN; ++j) {
                            const f16x8_t yh = half_values(y[j][2 * h], y[j][2 * h + 1]);
#pragma unroll
                            for (int i = 0; i < T::SM; ++i)
                                d[j][i] = __builtin_amdgcn_mfma_f32_32x32x16_f16(yh, xh[i], q + h == 0 ? f32x16_t{} : d[j][i], 0, 0, 0);
                        }
                    }
                }
#pragma unroll
                for (int j = 0; j < T::SN; ++j)
#pragma unroll
                    for (int i = 0; i < T::SM; ++i) add_step(stage, step, d[j][i], j, i, sa[i]);
            } else {
                i32x8_t x[T::SM][2];
#pragma unroll
                for (int i = 0; i < T::SM; ++i) x[i][0] = operand(rows_x, i, 0), x[i][1] = operand(rows_x, i, 1);
#pragma unroll
                for (int j = 0; j < T::SN; ++j) {
                    const i32x8_t y0 = operand(rows_w, j, 0), y1 = operand(rows_w, j, 1);
#pragma unroll
                    for (int i = 0; i < T::SM; ++i) {
                        f32x16_t d = product_f8(y0, x[i][0], f32x16_t{});
                        d = product_f8(y1, x[i][1], d);
                        add_step(stage, step, d, j, i, sa[i]);
                    }
                }
            }
        }
    }
    // the loads past the end are done, and every wave has read its last stage
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();
    float* mine = reinterpret_cast<float*>(lds) + w * T::TM * T::PITCH;
#pragma unroll
    for (int piece = 0; piece < T::TN / T::PW; ++piece) {
#pragma unroll
        for (int j = 0; j < T::PW / 32; ++j)
#pragma unroll
            for (int i = 0; i < T::SM; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16_t& d = acc[piece * (T::PW / 32) + j][i];
                    *reinterpret_cast<float4*>(mine + (32 * i + (lane & 31)) * T::PITCH + 32 * j + 8 * q + 4 * ((lane >> 5) & 1)) =
                        float4{d[4 * q], d[4 * q + 1], d[4 * q + 2], d[4 * q + 3]};
                }
        __builtin_amdgcn_wave_barrier();                 // the wave's own LDS operations stay in order
        constexpr int ACROSS = T::PW / 8;                // lanes of a row
#pragma unroll
        for (int i = 0; i < T::TM * ACROSS / 64; ++i) {
            const int r = (i * 64 + lane) / ACROSS, c = (lane % ACROSS) * 8;
            const int64_t row = m0 + wm * T::TM + r, col = n0 + wn * T::TN + piece * T::PW + c;
            if (row >= p.m || col >= p.n) continue;
            float v[8];
            load8<true>(mine, (size_t)r * T::PITCH + c, v);
            if (p.splits > 1) {
                store8<true>(p.parts, ((size_t)split * p.m + row) * p.n + col, v);
                continue;
            }
            if (p.add) {
                float o[8];
                load8<EXACT>(p.add, row * p.add_stride + col, o);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += o[e];
            }
            store8<EXACT>(p.out, row * p.out_stride + col, v);
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Adds the parts of the sums, in order, and `add`.
template <bool F32>
__global__ void __launch_bounds__(256) moe_product_join(ProductArgs p) {
    const int across = p.n / 8;
    const int64_t items = (int64_t)p.m * across;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < items; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / across;
        const int col = (int)(i - row * across) * 8;
        float v[8] = {};
        for (int s = 0; s < p.splits; ++s) {
            float o[8];
            load8<true>(p.parts, ((size_t)s * p.m + row) * p.n + col, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        if (p.add) {
            float o[8];
            load8<F32>(p.add, row * p.add_stride + col, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        store8<F32>(p.out, row * p.out_stride + col, v);
    }
}

namespace {

using Wide = Tile<256, 256, 4, 2, 2>;
using Mid = Tile<128, 128, 2, 2, 2>;
using Low = Tile<64, 128, 1, 4, 3>;

enum Kind { WIDE, MID, LOW };

struct Plan {
    Kind kind;
    int splits;
};

int64_t tiles_of(int m, int n, int bm, int bn) { return (int64_t)((m + bm - 1) / bm) * ((n + bn - 1) / bn); }

Plan plan(int m, int n, int k, bool f32) {
    const int steps = k / BK;
    Plan p;
    int64_t tiles;
    if (m <= 64) p.kind = LOW, tiles = tiles_of(m, n, 64, 128);
    else if (!f32 && tiles_of(m, n, 256, 256) >= 256) p.kind = WIDE, tiles = tiles_of(m, n, 256, 256);
    else p.kind = MID, tiles = tiles_of(m, n, 128, 128);
    p.splits = 1;
    if (p.kind != WIDE && tiles < 256 && steps > 1) {
        p.splits = (int)((512 + tiles - 1) / tiles);
        if (p.splits > 16) p.splits = 16;
        if (p.splits > steps) p.splits = steps;
    }
    return p;
}

template <typename T, bool EXACT, bool ROWS>
void go(const ProductArgs& p, hipStream_t stream) {
    const int64_t blocks = tiles_of(p.m, p.n, T::BM, T::BN) * p.splits;
    hipLaunchKernelGGL((moe_product<T, EXACT, ROWS>), dim3((unsigned)blocks), dim3(T::NT),
                       (unsigned)T::template lds<ROWS>(), stream, p);
}

template <bool EXACT, bool ROWS>
void go(Kind kind, const ProductArgs& p, hipStream_t stream) {
    if (kind == LOW) go<Low, EXACT, ROWS>(p, stream);
    else if (kind == MID) go<Mid, EXACT, ROWS>(p, stream);
    else if constexpr (!EXACT) go<Wide, EXACT, ROWS>(p, stream);
}

}  // namespace

int64_t product_workspace(int m, int n, int k, int b_scale, int out_type) {
    if (m == 0 || n == 0) return 0;
    const Plan q = plan(m, n, k, out_type == MEGA_MOE_F32);
    return q.splits > 1 ? (int64_t)q.splits * m * n * 4 : 0;
}

void launch_product(const mega_moe_product_args& g, hipStream_t stream) {
    const bool f32 = g.out_type == MEGA_MOE_F32, rows = g.b_scale == MEGA_MOE_SCALE_ROW;
    const Plan q = plan(g.m, g.n, g.k, f32);
    const ProductArgs p = {g.a, g.b, g.a_sf, g.b_sf, g.add, g.out, static_cast<float*>(g.workspace), g.a_stride, g.b_stride,
                           g.a_sf_stride, g.b_sf_stride, g.add_stride, g.out_stride, g.m, g.n, g.k / BK, q.splits};
    if (f32) rows ? go<true, true>(q.kind, p, stream) : go<true, false>(q.kind, p, stream);
    else rows ? go<false, true>(q.kind, p, stream) : go<false, false>(q.kind, p, stream);
    if (q.splits > 1) {
        const int64_t n = ((int64_t)g.m * (g.n / 8) + 255) / 256;
        const dim3 grid((unsigned)(n < 65536 ? n : 65536));
        if (f32) hipLaunchKernelGGL(moe_product_join<true>, grid, dim3(256), 0, stream, p);
        else hipLaunchKernelGGL(moe_product_join<false>, grid, dim3(256), 0, stream, p);
    }
}

}  // namespace mega_moe
