// out = a . b^T + add of E4M3 codes with float scales for 128 columns: of a's
// rows, and of b's rows or 128 x 128 blocks.
#include <hip/hip_runtime.h>

#include "block_util.h"
#include "product.h"

namespace mega_moe {

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
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
// that a load instruction covers eight whole rows and an operand's reads meet
// distinct banks. A wave's 16-byte reads are served 16 lanes at a time, lanes 0-3, 12-15,
// 20-27 and then 4-11, 16-19, 28-31 of each half: rows 0-3 and 12-15 of one chunk go with
// rows 4-11 of the next, so that these have the upper four places of their chunk and those the lower
// four. (With row ^ row / 8 % 2 half of the reads' cycles were conflicts.)
__device__ __forceinline__ int turn(int row) {
    return (((row >> 2) ^ (row >> 3)) & 1) << 2 | ((row >> 3) & 1) << 1 | ((row >> 1) & 1);
}

// The operand of 16 rows (slice s) of a step: lane r + 16 g has row r, chunks g and
// g + 4 (alike for a and b).  Every read of a stage is one of integers: of other types the
// compiler would wait for all loads into LDS first.
__device__ __forceinline__ i32x8_t operand(const uint8_t* rows, int s) {
    const int r = threadIdx.x & 15, g = (threadIdx.x >> 4) & 3;
    const uint8_t* row = rows + (16 * s + r) * BK;
    const i32x4_t lo = *reinterpret_cast<const i32x4_t*>(row + 16 * (g ^ turn(r)));
    const i32x4_t hi = *reinterpret_cast<const i32x4_t*>(row + 16 * ((g + 4) ^ turn(r)));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Eight codes as F16: exact.
__device__ __forceinline__ f16x8_t half_values(int lo, int hi) {
    const f16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const f16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const f16x2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const f16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    return f16x8_t{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// An operand as the matrix instructions take it, and its products with another's:
// 16 x 16 x 128, in one instruction or in four that follow each other.
template <bool EXACT>
struct Ready {
    static constexpr int N = 1;
    i32x8_t v;
    Ready() = default;
    __device__ __forceinline__ explicit Ready(const i32x8_t& raw) : v(raw) {}
    __device__ __forceinline__ f32x4_t times(const Ready& o, int, const f32x4_t& c) const {
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(v, o.v, c, 0, 0, 0, 0, 0, 0);   // scales 0: none
    }
};

template <>
struct Ready<true> {
    static constexpr int N = 4;
    f16x8_t v[4];
    Ready() = default;
    __device__ __forceinline__ explicit Ready(const i32x8_t& raw) {
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = half_values(raw[2 * q], raw[2 * q + 1]);
    }
    __device__ __forceinline__ f32x4_t times(const Ready& o, int q, const f32x4_t& c) const {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(v[q], o.v[q], c, 0, 0, 0);
    }
};

// Tiles.  BM x BN results, by WK groups of WM x WN waves: a group has every WK-th
// step, and the groups' sums meet at the end.  S rounds (a step of every group) in LDS.
template <int BM_, int BN_, int WM_, int WN_, int WK_, int S_>
struct Tile {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, WK = WK_, S = S_;
    static constexpr int NW = WM * WN, NT = 64 * NW * WK;  // NW: of a group
    static constexpr int TM = BM / WM, TN = BN / WN;       // a wave's
    static constexpr int SM = TM / 16, SN = TN / 16;
    static constexpr int A_LOADS = BM / 8 / NW, B_LOADS = BN / 8 / NW;     // of 1 KB, of a wave and step
    static constexpr int LOADS = A_LOADS + B_LOADS;
    static constexpr int OFF_B = BM * BK, STAGE = OFF_B + BN * BK;         // of a group
    static constexpr int ROUND = STAGE * WK;
    // behind the rounds the scales of eight steps, twice: [row][step] of a, [8 rows][step][row] of b, or
    // [128 rows][step] (and zeros behind them, as far as a load goes)
    static constexpr int OFF_SFA = S * ROUND, SFA = BM * 32, OFF_SFB = OFF_SFA + 2 * SFA, SFB = BN * 32;
    // two rounds of the widest tile fill LDS; each wave's first columns of b are the even blocks of loads
    static constexpr bool EARLY = SN >= 8 && S == 2 && TN / 2 == 8 * NW;
    static constexpr int PITCH = TN + 4;                 // of the groups' sums, which meet in LDS
    template <bool ROWS>
    static constexpr int lds() {
        const int a = OFF_SFB + 2 * (ROWS ? SFB : 256), b = WK == 1 ? 0 : WK * NW * TM * PITCH * 4;
        return a > b ? a : b;
    }
    static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "loads");
    static_assert((8 * NW) % 16 == 0, "turn() is the same for a wave's rows");
    static_assert(TN == 128 || 128 % TN == 0, "one block of scales to a wave");
    static_assert(SN >= 2 && SN % 2 == 0, "two columns are read ahead, and leave together");
    static_assert(8 % WK == 0 && WK < 8, "scales of eight steps last for whole rounds, and two or more");
    static_assert(8 / WK >= S - 1, "the next scales are older than the loads that meet() leaves in flight");
    static_assert(lds<true>() <= 160 * 1024, "LDS");
};

// What workgroup `id` of `total` computes: the runs of ids that go to one of the
// eight dies (id % 8) are neighbours in the order.
__device__ __forceinline__ int in_order(int id, int total) {
    const int die = id & 7, q = total >> 3, r = total & 7;
    return die * q + (die < r ? die : r) + (id >> 3);
}

}  // namespace

// One tile, or one of `splits` parts of its steps.  Per step of 128 columns the matrix unit sums codes'
// products, and the result times the two scales is added to the tile in float32.  b's rows are the
// matrix instruction's first operand, a's the second, so that a lane has one row of
// a result (16 of a slice) and register v column 4 (lane / 16) + v: the scale of
// a's row is one value for a lane.
//
// A round's barrier lies before its last two columns of blocks, whose operands are in
// registers by then: behind it the round's place in LDS is free for new loads,
// and the next round's operands are read while the matrix unit has those columns.
//
// What bounds it: with few rows what a compute unit takes in, some 40 to 65 KB/us of operands (deeper
// rounds, more waves, or fewer bytes of b and more of a, change nothing), so that small tiles, all compute units
// and no second launch are best: 128 x 7168 x 4096 11.9 us, 128 x 2048 x 7168 7.4. With many rows the matrix
// unit (busy for 60% of the cycles) and the scaling's vector instructions (39%; both for 27%), which share the issue,
// and the card's power: 8192 x 7168 x 4096 197 to 211 us by the card (2.3 to 2.45 PFLOP/s; a library product of the same
// codes with one scale, on a card where this one takes 200 to 206, 157 at first and 202 once it is warm). F32 results:
// four F16 instructions (twice the FP8's time in all) behind 16 conversions for each operand; 4096 x 4096 x 2048 with
// scales of rows 68 to 74 us (1.0 PFLOP/s).
template <typename T, bool EXACT, bool ROWS>
__global__ void __launch_bounds__(T::NT) moe_product(ProductArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    constexpr int S = T::S, LOADS = T::LOADS, ROUND = T::ROUND;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int group = wave / T::NW, w = wave % T::NW;
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
    const int rounds = (steps + T::WK - 1) / T::WK;

    const int rows_a = (int)min((int64_t)T::BM, p.m - m0), rows_b = (int)min((int64_t)T::BN, p.n - n0);
    const uint8_t* const a0 = p.a + m0 * p.a_stride + (int64_t)step0 * BK;
    const uint8_t* const b0 = p.b + n0 * p.b_stride + (int64_t)step0 * BK;
    const float* const a_sf0 = p.a_sf + m0 * p.a_sf_stride + step0;
    const float* const b_sf0 = p.b_sf + (ROWS ? n0 : n0 / 128) * p.b_sf_stride + step0;
    const int rows_sfb = ROWS ? rows_b : (rows_b + 127) / 128;
    const uint32_t bytes_a = (uint32_t)((rows_a - 1) * p.a_stride + (int64_t)steps * BK);
    const uint32_t bytes_b = (uint32_t)((rows_b - 1) * p.b_stride + (int64_t)steps * BK);
    const uint32_t bytes_sfa = (uint32_t)((rows_a - 1) * p.a_sf_stride + steps) * 4;
    const uint32_t bytes_sfb = (uint32_t)((rows_sfb - 1) * p.b_sf_stride + steps) * 4;
    // a wave's rows of a step: 8 (NW j + w) + lane / 8, and the chunk that belongs to lane % 8;
    // rows behind the last lie beyond the buffer by this offset alone
    const int r8 = 8 * w + (lane >> 3);
    const int voff_a = r8 * (int)p.a_stride + 16 * ((lane & 7) ^ turn(r8));
    const int voff_b = r8 * (int)p.b_stride + 16 * ((lane & 7) ^ turn(r8));
    const int jump_a = 8 * T::NW * (int)p.a_stride, jump_b = 8 * T::NW * (int)p.b_stride;

    // Load `part` (of LOADS) of the group's step of a round; past the last step the same
    // instructions, on buffers of no bytes: LDS gets zeros.
    const auto issue = [&](int place, int round, int part) {
        uint8_t* stage = lds + place + group * T::STAGE;
        const int step = round * T::WK + group;
        const uint32_t real = step < steps ? ~0u : 0u;
        if (part < T::A_LOADS) {
            load16_lds(buffer(a0, bytes_a & real), stage + (T::NW * part + w) * 1024, voff_a + part * jump_a, step * BK);
        } else {
            const int j = part - T::A_LOADS;
            load16_lds(buffer(b0, bytes_b & real), stage + T::OFF_B + (T::NW * j + w) * 1024, voff_b + j * jump_b, step * BK);
        }
    };
    // The scales of steps [8 chunk, 8 chunk + 8), eight rows to an instruction: step by step each would
    // be a line of its own, half as many again as the codes' (which cost the widest tile 6%, 128 x 128 12%).
    // 0 behind the last step.
    const auto load_scales = [&](int chunk) {
        // lanes are [row][step] of a's eight rows and steps, [step][row] of b's, whose scales are read by rows
        const auto rows_of = [&](const float* base, uint32_t bytes, int stride, int rows, uint8_t* to, int row, int step) {
            const bool real = chunk * 8 + step < steps;
#pragma unroll
            for (int b = 0; b < (rows / 8 + T::NT / 64 - 1) / (T::NT / 64); ++b) {
                const int block = b * (T::NT / 64) + wave;
                if (rows / 8 % (T::NT / 64) && block >= rows / 8) break;
                load4_lds(buffer(base, bytes), to + block * 256, real ? ((8 * block + row) * stride + step) * 4 : 0x7fffff00, chunk * 32);
            }
        };
        rows_of(a_sf0, bytes_sfa, (int)p.a_sf_stride, T::BM, lds + T::OFF_SFA + (chunk & 1) * T::SFA, lane >> 3, lane & 7);
        if constexpr (ROWS)
            rows_of(b_sf0, bytes_sfb, (int)p.b_sf_stride, T::BN, lds + T::OFF_SFB + (chunk & 1) * T::SFB, lane & 7, lane >> 3);
        else if (wave == 0)
            rows_of(b_sf0, bytes_sfb, (int)p.b_sf_stride, 8, lds + T::OFF_SFB + (chunk & 1) * 256, lane >> 3, lane & 7);
    };

    f32x4_t acc[T::SN][T::SM];
#pragma unroll
    for (int j = 0; j < T::SN; ++j)
#pragma unroll
        for (int i = 0; i < T::SM; ++i) acc[j][i] = f32x4_t{};

    // where the wave's rows of a stage are, and its scales
    const int at_x = group * T::STAGE + wm * T::TM * BK, at_y = group * T::STAGE + T::OFF_B + wn * T::TN * BK;
    const int at_sa = T::OFF_SFA + (wm * T::TM + (lane & 15)) * 32, at_sb = T::OFF_SFB + (wn * T::TN + (lane >> 5) * 8) * 32 + (lane >> 4 & 1) * 16;
    // b's block of scales is one for the wave (tiles start and end with blocks, or within one)
    const auto block_scale = [&](int step) {
        if constexpr (ROWS) return 1.0f;
        else return __int_as_float(*reinterpret_cast<const int*>(lds + T::OFF_SFB + (step >> 3 & 1) * 256 + (step & 7) * 4 + wn * T::TN / 128 * 32));
    };
    const auto row_scale = [&](int step, int i) {
        return __int_as_float(*reinterpret_cast<const int*>(lds + (step >> 3 & 1) * T::SFA + (step & 7) * 4 + at_sa + 16 * i * 32));
    };
    const auto column_scales = [&](int step, int j) {
        return *reinterpret_cast<const i32x4_t*>(lds + (step >> 3 & 1) * T::SFB + (step & 7) * 32 + at_sb + 16 * j * 32);
    };
    // With wide tiles, whose two rounds fill LDS, what of a round's place is read first takes new loads half a
    // round earlier: a's rows, and the rows of b's first columns (loads 0, 2, .. of b).
    constexpr bool EARLY = T::EARLY;
    constexpr int FIRST = EARLY ? T::A_LOADS + T::B_LOADS / 2 : 0;
    const auto order = [&](int n) {                      // of the loads
        if (!EARLY || n < T::A_LOADS) return n;
        return n < FIRST ? T::A_LOADS + 2 * (n - T::A_LOADS) : T::A_LOADS + 2 * (n - FIRST) + 1;
    };
    // This wave's loads of the next round are there and its reads of this one done, then every wave's.  (Scales
    // loaded since are older than the loads that are left in flight: they are waited for too.)
    const auto meet = [&]() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S - 2) * LOADS + FIRST) : "memory");
    };
    // the reads of a's rows and of b's first columns are done
    const auto meet_early = [&]() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

    if (steps > 0) {
        load_scales(0);
#pragma unroll
        for (int i = 0; i < S; ++i)
#pragma unroll
            for (int n = 0; n < LOADS; ++n) issue(i * ROUND, i, order(n));
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((S - 1) * LOADS) : "memory");
        int place = 0, step = group;
        float sa[T::SM], sb = block_scale(step);
        i32x8_t x_raw[T::SM], y_raw[2] = {operand(lds + at_y, 0), operand(lds + at_y, 1)};
        i32x4_t cs_next = {};
        if constexpr (ROWS) cs_next = column_scales(step, 0);
#pragma unroll
        for (int i = 0; i < T::SM; ++i) {
            x_raw[i] = operand(lds + at_x, i);
            sa[i] = row_scale(step, i);
        }
        for (int round = 0; round < rounds; ++round, step += T::WK) {
            const int next = place + ROUND == S * ROUND ? 0 : place + ROUND;
            // the next eight steps' scales, in the place of the last eight's
            if (round * T::WK % 8 == 0) load_scales(round * T::WK / 8 + 1);
            // while the matrix unit has the next blocks, those before them are added: EXACT by whole
            // columns of blocks, whose chains of four go on side by side, else three blocks later
            constexpr int BEHIND = EXACT ? T::SM : 3, RING = EXACT ? 2 * T::SM : 4, BLOCKS = T::SN * T::SM;
            f32x4_t d[RING];
            float s[T::SM];
            i32x4_t cs[T::SN];
            cs[0] = cs_next;
            const auto add_block = [&](int n) {
                const int j = n / T::SM, i = n % T::SM;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    acc[j][i][e] = fmaf(d[n % RING][e], ROWS ? s[i] * __int_as_float(cs[j][e]) : s[i], acc[j][i][e]);
            };
#pragma unroll
            for (int i = 0; i < T::SM; ++i) s[i] = sa[i] * sb;
            Ready<EXACT> x[T::SM];
#pragma unroll
            for (int i = 0; i < T::SM; ++i) x[i] = Ready<EXACT>(x_raw[i]);
#pragma unroll
            for (int j = 0; j < T::SN; ++j) {
                const Ready<EXACT> y(y_raw[0]);
                if constexpr (ROWS && T::SN == 2) {
                    if (j == 0) cs[1] = column_scales(step, 1);
                }
                // the round's last reads were those of two columns ahead
                if (EARLY && j == 2) meet_early();
                if (j == T::SN - 2) meet();
                const int from = j + 2 < T::SN ? place : next, ahead = (j + 2) % T::SN;
                y_raw[0] = y_raw[1];
                y_raw[1] = operand(lds + from + at_y, ahead);
                // b's scales a column ahead, the last column's before the barrier
                if constexpr (ROWS) {
                    if (j + 2 < T::SN) cs[j + 1] = column_scales(step, j + 1);
                    if (j + 3 == T::SN) cs[j + 2] = column_scales(step, j + 2);
                    if (j + 1 == T::SN) cs_next = column_scales(step + T::WK, 0);
                }
                // The new loads one by one between the last columns' instructions: one after the other they
                // would hold up every wave for as long as the loads take.
                // (the early ones over the four columns up to the second barrier's, the others over two)
                const bool early = EARLY && j >= 2 && j < T::SN - 2, late = j >= T::SN - 2;
                const int before = (early ? j - 2 : j - (T::SN - 2)) * T::SM * Ready<EXACT>::N;
                const auto load_some = [&](int slot) {
                    const int lo = early ? 0 : FIRST, hi = early ? FIRST : LOADS;
                    const int slots = (early ? T::SN - 4 : 2) * T::SM * Ready<EXACT>::N;
#pragma unroll
                    for (int n = lo; n < hi; ++n)
                        if ((n - lo) * slots / (hi - lo) == before + slot) issue(place, round + S, order(n));
                };
                // (the scales a column before the operands: what the next round waits for first)
                if (j == T::SN - 2) {
#pragma unroll
                    for (int i = 0; i < T::SM; ++i) sa[i] = row_scale(step + T::WK, i);
                    sb = block_scale(step + T::WK);
                }
                const auto read_next = [&](int i) { x_raw[i] = operand(lds + next + at_x, i); };
                if constexpr (EXACT) {
#pragma unroll
                    for (int q = 0; q < Ready<EXACT>::N; ++q)
#pragma unroll
                        for (int i = 0; i < T::SM; ++i) {
                            f32x4_t& o = d[(j * T::SM + i) % RING];
                            o = y.times(x[i], q, q == 0 ? f32x4_t{} : o);
                            if (early || late) {
                                __builtin_amdgcn_sched_barrier(0);
                                load_some(q * T::SM + i);
                                __builtin_amdgcn_sched_barrier(0);
                            }
                        }
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < T::SM; ++i) {
                        if (j + 1 == T::SN) read_next(i);
                        if (j > 0) add_block((j - 1) * T::SM + i);
                    }
                    __builtin_amdgcn_sched_barrier(0);
                } else {
#pragma unroll
                    for (int i = 0; i < T::SM; ++i) {
                        const int n = j * T::SM + i;
                        d[n % RING] = y.times(x[i], 0, f32x4_t{});
                        __builtin_amdgcn_sched_barrier(0);
                        if (early || late) load_some(i);
                        if (j + 1 == T::SN) read_next(i);
                        if (n >= BEHIND) add_block(n - BEHIND);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                }
            }
#pragma unroll
            for (int n = BLOCKS > BEHIND ? BLOCKS - BEHIND : 0; n < BLOCKS; ++n) add_block(n);
            place = next;
        }
    }
    const bool adds = p.add && p.splits == 1;
    const auto load_add = [&](int64_t row, int64_t col, u32x4_t (&o)[EXACT ? 2 : 1]) {
        const bool real = adds && row < p.m && col < p.n;
#pragma unroll
        for (int h = 0; h < (EXACT ? 2 : 1); ++h) o[h] = real ? raw8<EXACT>(p.add, row * p.add_stride + col)[h] : u32x4_t{0u, 0u, 0u, 0u};
    };
    // Eight results of a row leave the lane that has them.
    const auto leave = [&](int64_t row, int64_t col, float (&v)[8], const u32x4_t (&add)[EXACT ? 2 : 1]) {
        if (row >= p.m || col >= p.n) return;
        if (p.splits > 1) {
            store8<true>(p.parts, ((size_t)split * p.m + row) * p.n + col, v);
            return;
        }
        if (adds) {
            float o[8];
            values8<EXACT>(add, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        store8<EXACT>(p.out, row * p.out_stride + col, v);
    };
    // the loads past the end are done: LDS is the workgroup's until then
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    if constexpr (T::WK == 1) {
        // A lane has four columns of a block; two blocks side by side give it eight of one, whose 16 rows' stores
        // are 64 bytes or more each. (Through LDS, in whole lines, 8192 x 7168 x 4096 takes 1% less, but 8192 x 2048
        // x 7168 with an addend 172 us, not 162, and 4096 x 512 x 4096 with F32 results 34.5, not 32.4.)
        const int g = lane >> 4;
        const int64_t row0 = m0 + wm * T::TM + (lane & 15), col0 = n0 + wn * T::TN + (g & 1) * 16 + (g >> 1) * 8;
        // (the addend a row of blocks ahead of the stores: it may be the output itself, whose stores its loads wait for)
        u32x4_t add[2][T::SN / 2][EXACT ? 2 : 1];
        const auto load_row = [&](int i) {
#pragma unroll
            for (int j = 0; j < T::SN; j += 2) load_add(row0 + 16 * i, col0 + 16 * j, add[i & 1][j / 2]);
        };
        if (adds) load_row(0);
#pragma unroll
        for (int i = 0; i < T::SM; ++i) {
            if (adds && i + 1 < T::SM) load_row(i + 1);
#pragma unroll
            for (int j = 0; j < T::SN; j += 2) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[j][i][e]), __float_as_uint(acc[j + 1][i][e]), false, false);
                    v[e] = __uint_as_float(x[0]);
                    v[4 + e] = __uint_as_float(x[1]);
                }
                leave(row0 + 16 * i, col0 + 16 * j, v, add[i & 1][j / 2]);
            }
        }
        return;
    }
    __syncthreads();                                     // every wave has read its last stage
    // a group's wave has TM x TN sums in LDS; the groups' are added in order
    float* tile = reinterpret_cast<float*>(lds);
    constexpr int OF_WAVE = T::TM * T::PITCH;
#pragma unroll
    for (int j = 0; j < T::SN; ++j)
#pragma unroll
        for (int i = 0; i < T::SM; ++i)
            *reinterpret_cast<f32x4_t*>(tile + wave * OF_WAVE + (16 * i + (lane & 15)) * T::PITCH + 16 * j + 4 * (lane >> 4)) = acc[j][i];
    __syncthreads();
    constexpr int ACROSS = T::TN / 8;                    // lanes of a row
    constexpr int ITEMS = T::TM * ACROSS, AT_ONCE = 64 * T::WK;
#pragma unroll 2
    for (int i = 0; i < (ITEMS + AT_ONCE - 1) / AT_ONCE; ++i) {
        const int r = ((i * T::WK + group) * 64 + lane) / ACROSS, c = (lane % ACROSS) * 8;
        if (ITEMS % AT_ONCE && r >= T::TM) continue;
        float v[8];
        load8<true>(tile + w * OF_WAVE, (size_t)r * T::PITCH + c, v);
#pragma unroll
        for (int g = 1; g < T::WK; ++g) {
            float o[8];
            load8<true>(tile + (g * T::NW + w) * OF_WAVE, (size_t)r * T::PITCH + c, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += o[e];
        }
        u32x4_t add[EXACT ? 2 : 1];
        load_add(m0 + wm * T::TM + r, n0 + wn * T::TN + c, add);
        leave(m0 + wm * T::TM + r, n0 + wn * T::TN + c, v, add);
    }
}

// Up to 16 rows of a: a workgroup has 16 rows of b over all of k, its W waves every W-th step each, from memory
// into registers, and their sums meet in LDS.  b is read once and by no other workgroup; a comes from
// the caches.  Memory bounds it.  Up to 256 workgroups (and with F32 results, whose operands fill the registers) 16
// waves of two steps at a time, and two ahead: 1 x 7168 x 4096 6.8 us, from HBM 7.6 (29 MB; eight waves of four steps
// 7.2 and 7.8). More of them two to a compute unit, of eight waves of three steps: 1 x 7168 x 18432 from HBM
// 25.8 us (5.1 TB/s; 16 waves 29.5). Loads of b past the caches took 10% longer, whole lines of
// eight rows to a load 5%. 16 rows read as much of a as of b, and large n goes to the tiles then (18432:
// 42 us against 31).
template <bool EXACT, bool ROWS, bool PAIRED>
__global__ void __launch_bounds__(PAIRED ? 512 : 1024, 4) moe_product_few(ProductArgs p) {
    constexpr int W = PAIRED ? 8 : 16, U = PAIRED ? 3 : 2, PITCH = 20;
    __shared__ __attribute__((aligned(16))) float sums[W][16][PITCH];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int rows_b = (int)min((int64_t)16, p.n - n0);
    const __amdgpu_buffer_rsrc_t ra = buffer(p.a, (uint32_t)((p.m - 1) * p.a_stride + (int64_t)p.steps * BK));
    const __amdgpu_buffer_rsrc_t rb = buffer(p.b + n0 * p.b_stride, (uint32_t)((rows_b - 1) * p.b_stride + (int64_t)p.steps * BK));
    const __amdgpu_buffer_rsrc_t rsa = buffer(p.a_sf, (uint32_t)((p.m - 1) * p.a_sf_stride + p.steps) * 4);
    const __amdgpu_buffer_rsrc_t rsb = buffer(ROWS ? p.b_sf + n0 * p.b_sf_stride : p.b_sf + n0 / 128 * p.b_sf_stride,
                                              (uint32_t)((ROWS ? (rows_b - 1) * p.b_sf_stride : 0) + p.steps) * 4);
    // a lane has chunks g and g + 4 of a row's 128 bytes, alike for a and b
    const int voff_a = r * (int)p.a_stride + g * 16, voff_b = r * (int)p.b_stride + g * 16;
    const int voff_sa = r * (int)p.a_sf_stride * 4, voff_sb = ROWS ? r * (int)p.b_sf_stride * 4 : 0;
    struct Step {
        u32x4_t b[2], a[2];
        uint32_t sa, sb;
    };
    const auto fetch = [&](Step& s, int step) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            s.b[h] = __builtin_amdgcn_raw_buffer_load_b128(rb, voff_b + 64 * h, step * BK, 0);
            s.a[h] = __builtin_amdgcn_raw_buffer_load_b128(ra, voff_a + 64 * h, step * BK, 0);
        }
        s.sa = __builtin_amdgcn_raw_buffer_load_b32(rsa, voff_sa, step * 4, 0);
        if constexpr (ROWS) s.sb = __builtin_amdgcn_raw_buffer_load_b32(rsb, voff_sb, step * 4, 0);
    };
    typedef const __attribute__((address_space(4))) float* constants_t;
    const constants_t b_sf = (constants_t)(ROWS ? nullptr : p.b_sf + n0 / 128 * p.b_sf_stride);
    f32x4_t acc = f32x4_t{};
    const auto add_step = [&](const Step& s, int step) {
        const Ready<EXACT> y(__builtin_bit_cast(i32x8_t, __builtin_shufflevector(s.b[0], s.b[1], 0, 1, 2, 3, 4, 5, 6, 7)));
        const Ready<EXACT> x(__builtin_bit_cast(i32x8_t, __builtin_shufflevector(s.a[0], s.a[1], 0, 1, 2, 3, 4, 5, 6, 7)));
        f32x4_t d = f32x4_t{};
#pragma unroll
        for (int q = 0; q < Ready<EXACT>::N; ++q) d = y.times(x, q, d);
        const float sa = __uint_as_float(s.sa);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float sb = ROWS ? __shfl(__uint_as_float(s.sb), 4 * g + e) : b_sf[step];
            acc[e] = fmaf(d[e], sa * sb, acc[e]);
        }
    };
    // U steps in flight behind the U that are added
    Step now[U], next[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (w + W * u < p.steps) fetch(now[u], w + W * u);
    for (int step = w; step < p.steps; step += W * U) {
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (step + W * (U + u) < p.steps) fetch(next[u], step + W * (U + u));
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (step + W * u < p.steps) add_step(now[u], step + W * u);
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u];
    }
    *reinterpret_cast<f32x4_t*>(&sums[w][r][4 * g]) = acc;
    __syncthreads();
    // a thread has two columns of a row
    const int row = threadIdx.x >> 3, c = (threadIdx.x & 7) * 2;
    const int64_t col = n0 + c;
    if (row >= p.m || col >= p.n) return;
    float v[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < W; ++i) {
        v[0] += sums[i][row][c];
        v[1] += sums[i][row][c + 1];
    }
    if constexpr (EXACT) {
        if (p.add) {
            const float2 o = *reinterpret_cast<const float2*>(static_cast<const float*>(p.add) + row * p.add_stride + col);
            v[0] += o.x, v[1] += o.y;
        }
        *reinterpret_cast<float2*>(static_cast<float*>(p.out) + row * p.out_stride + col) = float2{v[0], v[1]};
    } else {
        if (p.add) {
            const uint32_t o = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.add) + row * p.add_stride + col);
            v[0] += __uint_as_float(o << 16), v[1] += __uint_as_float(o & 0xffff0000u);
        }
        *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row * p.out_stride + col) = bf16_pair(v[0], v[1]);
    }
}

// Adds the parts of the sums, in order, and `add`: a launch (2.8 us of a call), 0.23 us for each part that a thread adds and
// 8 bytes of each of its elements.
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

using Wide = Tile<256, 256, 4, 2, 1, 2>;
using WideExact = Tile<128, 256, 2, 4, 1, 2>; // in its place with F32 results: the conversions' registers
                                              // leave no room for 256 x 256 (4096 x 4096 x 2048: 68 us, Mid 72)
using Mid = Tile<128, 128, 2, 2, 1, 2>;       // two workgroups to a compute unit
using Long = Tile<128, 128, 4, 2, 1, 4>;      // one, of eight waves with three rounds in flight: only up to 256 tiles,
                                              // which have a compute unit each anyway (1024 x 7168 x 4096: 37 us, Mid
                                              // 42; from HBM 40 and 57; but 2048 x 7168 x 4096: 71 us, Mid 65)
using Tall = Tile<192, 128, 4, 2, 1, 3>;      // one (576 x 2048 x 7168: 16.6 us, Mid 18.4; 417 x 3328 x 10288 23.4 and 26.5)
using Half = Tile<64, 128, 2, 2, 2, 3>;       // one, of two groups of waves (512 x 7168 x 4096: 23.9 us, Pair 25.6)
using Pair = Tile<64, 64, 2, 2, 1, 3>;        // two or three workgroups
using Deep = Tile<64, 64, 2, 2, 2, 3>;        // one, of two groups of waves
using Strip = Tile<32, 64, 1, 2, 4, 3>;       // (128 x 7168 x 4096 from HBM: 16.4 us, Deep's halves 18.1)
using Low = Tile<32, 32, 2, 1, 4, 3>;

template <typename T, bool EXACT, bool ROWS>
void go(const ProductArgs& p, hipStream_t stream) {
    const int64_t blocks = product_tiles(p.m, p.n, T::BM, T::BN) * p.splits;
    hipLaunchKernelGGL((moe_product<T, EXACT, ROWS>), dim3((unsigned)blocks), dim3(T::NT),
                       (unsigned)T::template lds<ROWS>(), stream, p);
}

template <bool EXACT, bool ROWS>
void go(int kind, const ProductArgs& p, hipStream_t stream) {
    switch (kind) {
        case FEW: {
            const unsigned blocks = (unsigned)((p.n + 15) / 16);
            if (EXACT || blocks <= 256) hipLaunchKernelGGL((moe_product_few<EXACT, ROWS, false>), dim3(blocks), dim3(1024), 0, stream, p);
            else if constexpr (!EXACT) hipLaunchKernelGGL((moe_product_few<EXACT, ROWS, true>), dim3(blocks), dim3(512), 0, stream, p);
            break;
        }
        case LOW: go<Low, EXACT, ROWS>(p, stream); break;
        case DEEP: go<Deep, EXACT, ROWS>(p, stream); break;
        case PAIR: go<Pair, EXACT, ROWS>(p, stream); break;
        case MID: go<Mid, EXACT, ROWS>(p, stream); break;
        case STRIP:
            if constexpr (!EXACT) go<Strip, EXACT, ROWS>(p, stream);
            break;
        case HALF:
            if constexpr (!EXACT) go<Half, EXACT, ROWS>(p, stream);
            break;
        case TALL:
            if constexpr (!EXACT) go<Tall, EXACT, ROWS>(p, stream);
            break;
        case LONG:
            if constexpr (!EXACT) go<Long, EXACT, ROWS>(p, stream);
            break;
        default: go<std::conditional_t<EXACT, WideExact, Wide>, EXACT, ROWS>(p, stream);
    }
}

}  // namespace

int64_t product_workspace(const ProductPlan& plan, int m, int n) { return plan.splits > 1 ? (int64_t)plan.splits * m * n * 4 : 0; }

void launch_product(const mega_moe_product_args& g, const ProductPlan& plan, hipStream_t stream) {
    const bool f32 = g.out_type == MEGA_MOE_F32, rows = g.b_scale == MEGA_MOE_SCALE_ROW;
    const ProductArgs p = {g.a, g.b, g.a_sf, g.b_sf, g.add, g.out, static_cast<float*>(g.workspace), g.a_stride, g.b_stride,
                           g.a_sf_stride, g.b_sf_stride, g.add_stride, g.out_stride, g.m, g.n, g.k / BK, plan.splits};
    if (f32) rows ? go<true, true>(plan.kind, p, stream) : go<true, false>(plan.kind, p, stream);
    else rows ? go<false, true>(plan.kind, p, stream) : go<false, false>(plan.kind, p, stream);
    if (plan.splits > 1) {
        const int64_t n = ((int64_t)g.m * (g.n / 8) + 255) / 256;
        const dim3 grid((unsigned)(n < 65536 ? n : 65536));
        if (f32) hipLaunchKernelGGL(moe_product_join<true>, grid, dim3(256), 0, stream, p);
        else hipLaunchKernelGGL(moe_product_join<false>, grid, dim3(256), 0, stream, p);
    }
}

}  // namespace mega_moe
