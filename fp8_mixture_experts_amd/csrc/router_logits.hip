// The router's product, logits = x . w^T, and its gradients.
#include <hip/hip_runtime.h>

#include <type_traits>

#include "block_util.h"
#include "router_logits.h"

namespace mega_moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Eight floats as the sum of P BF16 vectors: each term is what is left, rounded
// to nearest.  Two leave 2^-17 of the value, three nothing (24 bits).  Finite
// values below BF16's largest; an infinity becomes NaN.
template <int P>
__device__ __forceinline__ void split_bf16(const float (&v)[8], u32x4_t (&p)[P]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float r0 = v[2 * i], r1 = v[2 * i + 1];
#pragma unroll
        for (int q = 0; q < P; ++q) {
            p[q][i] = bf16_pair(r0, r1);
            r0 -= __uint_as_float(p[q][i] << 16);
            r1 -= __uint_as_float(p[q][i] & 0xffff0000u);
        }
    }
}

// Small products.  A tile of up to 16 tokens x 16 experts per workgroup; its 16
// waves take the K steps in turn, straight from memory, and their sums meet in
// LDS.  What bounds it is how fast one compute unit takes in its rows (about 40
// GB/s, whatever the others do), so the tile is the one that leaves the fewest
// bytes to each (small_tile below).  What a smaller tile than 16 x 16 leaves of
// the matrix instruction's rows and columns are other slices of k: rows and
// columns of the same slice meet on its diagonal blocks, whose sums are added at
// the end.  So every lane has something to load, and a wave the loads of STEPS
// steps in flight.  128 x 7168 x 32: 14 us with whole tiles on 16 compute
// units, 8.0 with 4 x 4 on 256 and the rest of the instruction zero, 6.1 so; one
// token 5.4 and 4.2, with float32 weights 8.8 and 5.6.
template <bool WF32>
__global__ void __launch_bounds__(1024)
moe_router_logits(mega_moe_router_logits_args a, int tile_t, int tile_e) {
    // Few enough that two workgroups share a compute unit (64 registers): with 8
    // steps, and 7 with float32 weights, 1024 x 640 x 151 takes 8.4 and 14.7 us, so
    // 6.9 and 8.7, and 1 x 7168 x 32 as long.
    constexpr int STEPS = WF32 ? 2 : 4;
    __shared__ float part[16][16][17];
    __shared__ float sums[16][17];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int H = a.hidden, E = a.num_experts;
    const int e_tiles = (E + tile_e - 1) / tile_e;
    const int e0 = (int)(blockIdx.x % e_tiles) * tile_e;
    const int t0 = (int)(blockIdx.x / e_tiles) * tile_t;
    // `wide` rows and columns of the tile, `slices` of k
    const int wide = tile_t > tile_e ? tile_t : tile_e, slices = 16 / wide;
    const int r = lane & 15 & (wide - 1), k_lane = (lane & 15) / wide * 32 + (lane >> 4) * 8;
    const bool has_t = r < tile_t && t0 + r < a.num_tokens, has_e = r < tile_e && e0 + r < E;
    const uint16_t* x = a.x + (int64_t)(t0 + r) * a.x_stride + k_lane;
    const size_t w_row = (size_t)(e0 + r) * H + k_lane;
    const int chunk = 32 * slices;               // k of a wave's step
    const int left = H - k_lane;                 // k from this lane's first on
    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = wave * chunk; k0 < H; k0 += 16 * chunk * STEPS) {
        u32x4_t xv[STEPS], wv[STEPS][WF32 ? 2 : 1];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int k = k0 + s * 16 * chunk;
            const u32x4_t none = {0u, 0u, 0u, 0u};
            xv[s] = none;
#pragma unroll
            for (int i = 0; i < (WF32 ? 2 : 1); ++i) wv[s][i] = none;
            if (has_t && k < left) xv[s] = *reinterpret_cast<const u32x4_t*>(x + k);
            if (has_e && k < left) {
#pragma unroll
                for (int i = 0; i < (WF32 ? 2 : 1); ++i) wv[s][i] = raw8<WF32>(a.w, w_row + k)[i];
            }
        }
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const bf16x8_t xb = __builtin_bit_cast(bf16x8_t, xv[s]);
            if constexpr (WF32) {
                float w[8];
                values8<true>(wv[s], w);
                u32x4_t p[3];
                split_bf16<3>(w, p);
#pragma unroll
                for (int q = 2; q >= 0; --q)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, p[q]), xb, acc, 0, 0, 0);
            } else {
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wv[s][0]), xb, acc, 0, 0, 0);
            }
        }
    }
    // lane l holds experts 4 (l / 16) .. + 3 of token l % 16
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][lane & 15][(lane >> 4) * 4 + i] = acc[i];
    __syncthreads();
    // the waves' sums, then the slices'
    const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
    if (threadIdx.x < 256) {
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 16; ++w) s += part[w][row][col];
        sums[row][col] = s;
    }
    __syncthreads();
    if (row >= tile_t || col >= tile_e || t0 + row >= a.num_tokens || e0 + col >= E) return;
    float s = 0.0f;
    for (int i = 0; i < slices; ++i) s += sums[i * wide + row][i * wide + col];
    a.logits[(int64_t)(t0 + row) * a.logits_stride + e0 + col] = s;
}

// ---------------------------------------------------------------------------
// Tiles through LDS, for batches of tokens and for the gradients.
// C[m, n] = sum over k of A[m, k] B[n, k] on 32 x 32 x 16 BF16 matrix
// instructions, each operand as one BF16 plane or three whose products add
// into the same accumulators, the small ones first.  A float32 operand is split
// into its planes where its fragments are read.
//
// A workgroup computes BM x BN.  Steps of 64 k go from memory straight into
// LDS (16 bytes a lane, no registers), STAGES - 1 of them ahead
// of the one that is multiplied.  An operand lies in memory, and in LDS, in
// one of four ways:
//   k_major    rows of k: a fragment's eight k are one 16-byte read
//   k_float    the same in float32: two reads
//   row_major  k after k, each a row of m (or n): the LDS reads that turn
//              4 x 16 values around give four k of a lane's row at a time
//   row_float  the same in float32: eight reads of one value
// Lanes that point outside an operand read zeros.
//
// LDS holds 16-byte chunks in the order in which they are loaded; where a
// chunk comes from is permuted within its row, so that the reads of a fragment
// spread over all banks: in a k_major row r chunk c lies at c ^ (r / 2) % 8, in a
// k_float row at c ^ r % 16, in a row_float row at c ^ (r & 8); of a row_major row the
// pairs of chunks (16 columns, one turned read) are permuted by the bits in which the
// eight rows of a read differ.
// ---------------------------------------------------------------------------

enum class Lay { k_major, row_major, k_float, row_float };

struct Operand {
    const void* p;
    int64_t stride;        // elements from one row to the next, in memory
    int64_t rows, k;       // extents: of m or n, and of k (rows in memory: of m or n
                           // for k_major, of k for row_major)
};

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4a_t __attribute__((ext_vector_type(4), aligned(4)));
#define LDS_PTR __attribute__((address_space(3)))

constexpr int STEP = 64;                       // k of a step
constexpr uint32_t OUTSIDE = 0x7fffff00u;      // beyond every buffer's bytes

// `bytes` bytes at `base`; both are the same for the whole wave.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* base, int64_t bytes) {
    const uint64_t p = (uint64_t)(uintptr_t)base;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)p);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(p >> 32));
    const int n = __builtin_amdgcn_readfirstlane((int)(bytes < 0 ? 0 : bytes));
    return __builtin_amdgcn_make_buffer_rsrc((void*)(uintptr_t)((uint64_t)hi << 32 | lo), 0, n, 0x00020000);
}

// The pairs of chunks of a row_major row of R columns, permuted.
template <int R>
__device__ __forceinline__ int pair_swizzle(int row) {
    return R >= 128 ? (row & 3) | (row >> 1 & 4) : (row >> 1 & 1) | (row >> 2 & 2);
}

// One operand's planes of a step: R rows of m (or n) by STEP k.
template <Lay L, int P, int R, int THREADS>
struct Tile {
    static constexpr bool ROWS_OF_K = L == Lay::k_major || L == Lay::k_float;
    static constexpr bool FLOAT = L == Lay::k_float || L == Lay::row_float;
    static constexpr int SIZE = FLOAT ? 4 : 2, PER = 16 / SIZE;      // bytes of an element, elements of a chunk
    static constexpr int CHUNKS = R * STEP / PER;
    static constexpr int PER_LANE = CHUNKS / THREADS;    // loads per lane and step
    static constexpr int WIDTH = (ROWS_OF_K ? STEP : R) / PER;       // chunks of a row
    static_assert(CHUNKS % THREADS == 0, "whole loads");

    __device__ __forceinline__ static int swizzle(int r) {
        if constexpr (L == Lay::row_major) return pair_swizzle<R>(r) << 1;
        else if constexpr (L == Lay::k_float) return r & 15;
        else if constexpr (L == Lay::row_float) return r & 8;
        else return r >> 1 & 7;
    }

    // Byte offset of this lane's chunk of load i of a plane, from the tile's
    // first element, or OUTSIDE where its columns are.
    uint32_t at[PER_LANE];

    __device__ __forceinline__ void place(const Operand& o, int64_t row0) {
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
            const int id = i * THREADS + (int)threadIdx.x, r = id / WIDTH;
            const int c = (id % WIDTH) ^ swizzle(r);
            const bool in = ROWS_OF_K ? row0 + r < o.rows : row0 + c * PER < o.rows;
            at[i] = in ? (uint32_t)((r * o.stride + c * PER) * SIZE) : OUTSIDE;
        }
    }

    // Starts the loads of the step at k0; from k_end on, or the operand's own
    // end, they bring zeros.
    __device__ __forceinline__ void load(const Operand& o, int64_t row0, int64_t k0, int64_t k_end, u32x4_t* lds) const {
        const int64_t left = (k_end < o.k ? k_end : o.k) - k0;
        const int wave = threadIdx.x >> 6;
        // rows past the last lie outside of the buffer; chunks past the last k of
        // a row of k must be pointed there
        const int64_t n = ROWS_OF_K ? o.rows - row0 : left < STEP ? left : STEP;
        const int64_t width = ROWS_OF_K ? left : o.rows - row0;
        const int64_t first = ROWS_OF_K ? row0 * o.stride + k0 : k0 * o.stride + row0;
        const auto buf = buffer_of(static_cast<const char*>(o.p) + first * SIZE,
                                   left > 0 ? (((n < R ? n : R) - 1) * o.stride + width) * SIZE : 0);
#pragma unroll
        for (int i = 0; i < PER_LANE; ++i) {
            uint32_t off = at[i];
            if (ROWS_OF_K && left < STEP) {
                const int id = i * THREADS + (int)threadIdx.x;
                if (((id % WIDTH) ^ swizzle(id / WIDTH)) * PER >= left) off = OUTSIDE;
            }
            u32x4_t* to = lds + i * THREADS + __builtin_amdgcn_readfirstlane(wave) * 64;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(buf, (LDS_PTR void*)to, 16, (int)off, 0, 0, 0);
        }
    }

    // The fragment of rows r0 .. r0 + 31 and k 16 kk .. + 15 of a k_major tile:
    // lane l holds row r0 + l % 32, k 8 (l / 32) .. + 7 of them.
    __device__ __forceinline__ static bf16x8_t fragment(const u32x4_t* lds, int r0, int kk) {
        const int lane = threadIdx.x & 63, r = r0 + (lane & 31), c = kk * 2 + (lane >> 5);
        return __builtin_bit_cast(bf16x8_t, lds[r * WIDTH + (c ^ swizzle(r))]);
    }
    // The same of a float tile, split into its planes.
    __device__ __forceinline__ static void fragment(const u32x4_t* lds, int r0, int kk, bf16x8_t (&planes)[P]) {
        const int lane = threadIdx.x & 63, r = r0 + (lane & 31);
        float v[8];
        if constexpr (L == Lay::k_float) {
            const int c = kk * 4 + (lane >> 5) * 2;
            values8<true>(lds[r * WIDTH + (c ^ swizzle(r))], lds[r * WIDTH + ((c + 1) ^ swizzle(r))], v);
        } else {
            const int k = kk * 16 + (lane >> 5) * 8;     // eight k with the same swizzle
            const float* q = reinterpret_cast<const float*>(lds + k * WIDTH + (r / 4 ^ swizzle(k))) + r % 4;
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = q[i * WIDTH * 4];
        }
        u32x4_t p[P];
        split_bf16<P>(v, p);
#pragma unroll
        for (int i = 0; i < P; ++i) planes[i] = __builtin_bit_cast(bf16x8_t, p[i]);
    }

    // Of a row_major tile: where this lane's part of it starts, as an LDS byte
    // address, at kk = 0.  16 lanes turn a block of 4 k x 16 rows around: lane
    // i of them brings rows 4 (i % 4) .. + 3 of k i / 4 and takes row i; a
    // fragment is two such reads, of k 8 (l / 32) .. + 3 and of the next four.
    __device__ __forceinline__ static uint32_t turned_at(const u32x4_t* lds, int r0) {
        const int lane = threadIdx.x & 63, i = lane & 15, col = r0 + (lane >> 4 & 1) * 16 + (i & 3) * 4;
        const int row = (lane >> 5) * 8 + (i >> 2);
        const u32x4_t* chunk = lds + row * WIDTH + (col / 8 ^ swizzle(row));
        return (uint32_t)(uintptr_t)(LDS_PTR const void*)chunk + (col >> 2 & 1) * 8;
    }
    // Bytes on from there: to the next 16 k, and the other four k.
    static constexpr int NEXT_KK = 16 * WIDTH * 16, NEXT_HALF = 4 * WIDTH * 16;
};

// The turned reads of one kk, with the wait for them: the compiler would wait
// for the loads into LDS in flight before each.
typedef uint64_t Half;
__device__ __forceinline__ bf16x8_t halves(Half a, Half b) {
    struct Two { Half v[2]; };
    return __builtin_bit_cast(bf16x8_t, Two{{a, b}});
}

#define TURN(dst, at, off) "ds_read_b64_tr_b16 %" dst ", %" at " offset:%" off "\n\t"

// The two fragments at at1 and at2.
template <int OFF, int HALF>
__device__ __forceinline__ void turned(uint32_t at1, uint32_t at2, bf16x8_t (&f)[1][2]) {
    Half a, b, c, d;
    asm volatile(TURN("0", "4", "6") TURN("1", "4", "7") TURN("2", "5", "6") TURN("3", "5", "7")
                 "s_waitcnt lgkmcnt(0)"
                 : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d)
                 : "v"(at1), "v"(at2), "n"(OFF), "n"(OFF + HALF)
                 : "memory");
    f[0][0] = halves(a, b);
    f[0][1] = halves(c, d);
}

// Waits until this wave has at most N loads in flight, then for the others.
template <int N>
__device__ __forceinline__ void arrived() {
    static_assert(N < 64, "the counter's range");
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <typename F>
__device__ __forceinline__ void over_kk(F&& f) {
    static_assert(STEP == 64, "four instructions' k to a step");
    f(std::integral_constant<int, 0>{});
    f(std::integral_constant<int, 1>{});
    f(std::integral_constant<int, 2>{});
    f(std::integral_constant<int, 3>{});
}

// Where a product goes: float32 rows (the result, or one split's part of it in
// the workspace, [split][M][N]), or BF16 rows with something added.
struct Result {
    int64_t rows, cols;
    float* f32;
    int64_t stride;
    uint16_t* bf16;
    const uint16_t* add;
    int64_t add_stride;
};

// One product's operands, result and split of K.
struct Product {
    Operand a, b;
    Result out;
    int64_t k_split;
    int splits;
};

// The kind of a product, and what it needs of LDS (in chunks).
template <Lay LA_, int PA_, Lay LB_, int PB_, int BM_, int BN_, int STAGES_, bool OUT_BF16_, int WM_ = 2,
          int WN_ = 2>
struct Kind {
    static constexpr Lay LA = LA_, LB = LB_;
    static constexpr int PA = PA_, PB = PB_, BM = BM_, BN = BN_, STAGES = STAGES_;
    static constexpr int WM = WM_, WN = WN_, THREADS = WM * WN * 64;     // waves over the tile
    static constexpr bool OUT_BF16 = OUT_BF16_;
    static constexpr int PITCH = BN + 4;         // BF16 results go out through LDS, as rows of floats
    using TA = Tile<LA, PA, BM, THREADS>;
    using TB = Tile<LB, PB, BN, THREADS>;
    static constexpr int STAGE = TA::CHUNKS + TB::CHUNKS;
    static constexpr int OUT = OUT_BF16 ? BM * PITCH / 4 : 0;
    static constexpr int LDS = STAGE * STAGES > OUT ? STAGE * STAGES : OUT;
};

// Workgroup `block` of a product.
template <typename K>
__device__ __forceinline__ void product(u32x4_t* lds, const Product& x, unsigned block) {
    constexpr Lay LA = K::LA, LB = K::LB;
    constexpr int PA = K::PA, PB = K::PB, BM = K::BM, BN = K::BN, STAGES = K::STAGES, STAGE = K::STAGE, PITCH = K::PITCH;
    constexpr bool OUT_BF16 = K::OUT_BF16;
    constexpr int WM = K::WM, WN = K::WN, THREADS = K::THREADS;
    using TA = typename K::TA;
    using TB = typename K::TB;
    const Operand &A = x.a, &Bo = x.b;
    const Result& out = x.out;
    const int splits = x.splits;
    const int64_t k_split = x.k_split;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / WN * (TM * 32), wn = wave % WN * (TN * 32);
    const int n_tiles = (int)((Bo.rows + BN - 1) / BN);
    const int split = block % splits;
    const int64_t tile = block / splits;
    const int64_t m0 = tile / n_tiles * BM, n0 = tile % n_tiles * BN;
    const int64_t k_first = split * k_split;
    const int64_t k_end = k_first + k_split < A.k ? k_first + k_split : A.k;

    f32x16_t acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

    TA ta;
    TB tb;
    ta.place(A, m0);
    tb.place(Bo, n0);
    const auto load = [&](int64_t k0, int stage) {
        ta.load(A, m0, k0, k_end, lds + stage * STAGE);
        tb.load(Bo, n0, k0, k_end, lds + stage * STAGE + TA::CHUNKS);
    };
    constexpr int LOADS = TA::PER_LANE + TB::PER_LANE;
    // steps past the last load nothing but zeros, so that the count of loads in
    // flight is the same in every round
#pragma unroll
    for (int s = 0; s + 1 < STAGES; ++s) load(k_first + s * STEP, s);
    int stage = 0;
    for (int64_t k0 = k_first; k0 < k_end; k0 += STEP) {
        if constexpr (STAGES == 1) {
            load(k0, 0);
            arrived<0>();
        } else {
            // this step is there, and every wave has left the one before it,
            // whose place the newest load takes
            arrived<(STAGES - 2) * LOADS>();
            load(k0 + (STAGES - 1) * STEP, stage == 0 ? STAGES - 1 : stage - 1);
        }
        const u32x4_t* la = lds + stage * STAGE;
        const u32x4_t* lb = la + TA::CHUNKS;
        uint32_t at[2] = {0, 0};
        static_assert(LA != Lay::row_major, "only B is turned");
        if constexpr (LB == Lay::row_major) {
            static_assert(TN == 2 && PB == 1, "two fragments to a turned read");
            at[0] = TB::turned_at(lb, wn);
            at[1] = TB::turned_at(lb, wn + 32);
        }
        over_kk([&](auto step) {
            constexpr int kk = decltype(step)::value;
            bf16x8_t fa[PA][TM], fb[PB][TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) {
                bf16x8_t planes[PA];
                if constexpr (TA::FLOAT) TA::fragment(la, wm + i * 32, kk, planes);
                else planes[0] = TA::fragment(la, wm + i * 32, kk);
#pragma unroll
                for (int p = 0; p < PA; ++p) fa[p][i] = planes[p];
            }
            if constexpr (LB == Lay::row_major) {
                turned<kk * TB::NEXT_KK, TB::NEXT_HALF>(at[0], at[1], fb);
            } else {
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    bf16x8_t planes[PB];
                    if constexpr (TB::FLOAT) TB::fragment(lb, wn + j * 32, kk, planes);
                    else planes[0] = TB::fragment(lb, wn + j * 32, kk);
#pragma unroll
                    for (int p = 0; p < PB; ++p) fb[p][j] = planes[p];
                }
            }
            // the planes' products, the smallest first; beyond the last plane's
            // weight they are dropped
#pragma unroll
            for (int w = (PA > PB ? PA : PB) - 1; w >= 0; --w)
#pragma unroll
                for (int p = 0; p < PA; ++p) {
                    const int q = w - p;
                    if (q < 0 || q >= PB) continue;
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fb[q][j], fa[p][i], acc[i][j], 0, 0, 0);
                }
        });
        if constexpr (STAGES == 1) __syncthreads();
        else stage = stage + 1 == STAGES ? 0 : stage + 1;
    }

    arrived<0>();        // nothing is on its way into LDS any more
    // lane l holds row m = l % 32 and columns n = 8 g + 4 (l / 32) .. + 3, g < 4
    if constexpr (OUT_BF16) {
        float* rows = reinterpret_cast<float*>(lds);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    u32x4_t d;
#pragma unroll
                    for (int q = 0; q < 4; ++q) d[q] = __float_as_uint(acc[i][j][g * 4 + q]);
                    lds[((wm + i * 32 + (lane & 31)) * PITCH + wn + j * 32 + g * 8 + (lane >> 5) * 4) / 4] = d;
                }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < BM * BN / 8 / THREADS; ++i) {
            const int id = i * THREADS + (int)threadIdx.x;
            const int r = id / (BN / 8), c = id % (BN / 8) * 8;
            const int64_t m = m0 + r, n = n0 + c;
            if (m >= out.rows || n >= out.cols) continue;      // the rows come in eights
            float v[8];
            load8<true>(rows, (size_t)r * PITCH + c, v);
            if (out.add) {
                float d[8];
                load8<false>(out.add, m * out.add_stride + n, d);
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] += d[q];
            }
            store8<false>(out.bf16, m * out.stride + n, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int64_t m = m0 + wm + i * 32 + (lane & 31);
            if (m >= out.rows) continue;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int64_t n = n0 + wn + j * 32 + g * 8 + (lane >> 5) * 4;
                    if (n >= out.cols) continue;
                    float v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = acc[i][j][g * 4 + q];
                    float* o = out.f32 + (splits > 1 ? (split * out.rows + m) * out.cols : m * out.stride) + n;
                    if (n + 4 <= out.cols) {
                        u32x4a_t d;
#pragma unroll
                        for (int q = 0; q < 4; ++q) d[q] = __float_as_uint(v[q]);
                        *reinterpret_cast<u32x4a_t*>(o) = d;
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (n + q < out.cols) o[q] = v[q];
                    }
                }
        }
    }
}

// 8192 x 7168 x 256 with float32 weights: 90 to 97 us, 1.0 PFLOP/s of BF16 terms (a
// large library product reaches 1.44), with 9 us after it to add the parts of K;
// with BF16 weights 47 and 7 us (129 MB: 25 us), of which a compute unit takes in
// 1.8 MB at some 40 kB/us.
template <typename K>
__global__ void __launch_bounds__(K::THREADS)
moe_router_product(Product x) {
    __shared__ u32x4_t lds[K::LDS];
    product<K>(lds, x, blockIdx.x);
}

// Both gradients in one launch: workgroups of dw, which are few and long, and
// then those of dx, which fill up what is left.
// 4096 x 4096 x 64: 21 to 26 us (67 MB of x and dx: 13 us), and 4 us to add the parts
// of dw.  Larger tiles (64 x 256 for dw, for dx 64 x 256 or 128 x 128), which take in
// a quarter less, were slower (31 to 33 us in all against 26).  With dlogits and w
// split into planes beforehand, by a launch of their own, 28 us, and 15.5 us against
// 13.3 at 1024 x 2048 x 128.
template <typename KW, typename KX>
__global__ void __launch_bounds__(256)
moe_router_gradients(Product w, unsigned w_blocks, Product x) {
    __shared__ u32x4_t lds[KW::LDS > KX::LDS ? KW::LDS : KX::LDS];
    if (blockIdx.x < w_blocks) product<KW>(lds, w, blockIdx.x);
    else product<KX>(lds, x, blockIdx.x - w_blocks);
}

// Rows of `cols` floats as rows of `width`, a multiple of 4; columns behind the
// last are 0.
__global__ void __launch_bounds__(256)
moe_router_pad(const float* from, int64_t stride, int64_t rows, int cols, float* to, int width) {
    const int64_t units = width / 4, n = rows * units;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t r = i / units;
        const int c = (int)(i - r * units) * 4;
        const float* q = from + r * stride + c;
        u32x4_t v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = c + j < cols ? __float_as_uint(q[j]) : 0u;
        *reinterpret_cast<u32x4_t*>(to + r * width + c) = v;
    }
}

// Adds the splits' parts in order.
__global__ void __launch_bounds__(256)
moe_router_product_join(const float* ws, float* out, int64_t M, int64_t N, int64_t stride, int splits) {
    const int64_t total = M * N;
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < total; i += (int64_t)gridDim.x * 1024) {
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const int n = total - i < 4 ? (int)(total - i) : 4;
        for (int s = 0; s < splits; ++s) {
            const float* p = ws + s * total + i;
            if (n == 4) {
                const u32x4a_t d = *reinterpret_cast<const u32x4a_t*>(p);
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += __uint_as_float(d[q]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (q < n) v[q] += p[q];
            }
        }
        int64_t m = i / N, c = i - m * N;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (q >= n) break;
            out[m * stride + c] = v[q];
            if (++c == N) c = 0, ++m;
        }
    }
}

namespace {

constexpr int64_t MAX_TILE_STRIDE = 1 << 22;     // of floats: 128 rows within 32-bit byte offsets

struct Split {
    int n;               // parts of K
    int64_t k;           // K of a part, whole steps of 64
};

// Parts of K for a product of `tiles` tiles: enough for `want` workgroups, each
// with four steps or more.
Split split_for(int64_t tiles, int64_t K, int64_t want) {
    int n = 1;
    while (n < 16 && tiles * n < want && K / (2 * n) >= 256) n *= 2;
    const int64_t steps = (K + 63) / 64;
    return Split{n, (steps + n - 1) / n * 64};
}

int64_t tiles(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tile of a small product: the fewest bytes of rows for one compute unit of
// 256, in as many turns as the tiles take.
struct SmallTile {
    int t, e;
    int64_t bytes;       // for a compute unit, per k
};
SmallTile small_tile(const mega_moe_router_logits_args& a) {
    const int w_bytes = a.weight_type == MEGA_MOE_F32 ? 4 : 2;
    SmallTile best{16, 16, INT64_MAX};
    for (int t = 4; t >= 0; --t)
        for (int e = 4; e >= 0; --e) {
            const int64_t n = (int64_t)((a.num_tokens - 1 >> t) + 1) * ((a.num_experts - 1 >> e) + 1);
            const int64_t bytes = ((n - 1 >> 8) + 1) * ((2 << t) + (w_bytes << e));
            if (bytes < best.bytes) best = SmallTile{1 << t, 1 << e, bytes};
        }
    return best;
}

// Whether the 16 x 16 tiles compute the logits: one launch at about 40 kB/us for
// each compute unit, against one or two launches that read every row less often.
// They cross where a compute unit takes in about 300 kB and 20 rows of BF16:
// 16 x 16 and 128-row tiles at 1024 x 640 x 128 5.0 and 10.7 us (82 kB), 8192 x
// 640 x 31 8.5 and 9.5 (164 kB), 2048 x 7168 x 31 15.3 and 15.8 (459 kB), 4096 x
// 4096 x 31 17.2 and 16.5 (524 kB), 512 x 7168 x 512 51 and 19 (1.8 MB); with
// float32 weights 512 x 4096 x 128 14 and 18 (393 kB), 1024 x 1792 x 256 22 and 19
// (688 kB).
bool is_small(const mega_moe_router_logits_args& a, const SmallTile& s) {
    return s.bytes * a.hidden <= 300000 + 40 * a.hidden;
}

// The workspace: dlogits with whole chunks, then the parts of a split K.
struct Plan {
    Split split;
    int64_t parts, total;   // byte offset, and bytes in all
};

int64_t padded(int64_t E) { return (E + 3) / 4 * 4; }

int64_t forward_tiles(const mega_moe_router_logits_args& a) {
    const int64_t E = a.num_experts;
    return tiles(a.num_tokens, 128) * tiles(E, E <= 32 ? 32 : E <= 64 ? 64 : 128);
}

// Whether two workgroups share a compute unit: with float32 weights, where one
// each would leave parts of K longer than 2048.  In pairs and alone, us (part of K):
// 8192 x 7168 x 256 105 and 116, 16384 x 7168 x 128 107 and 117, 2048 x 7168 x 1024
// 95 and 100 (3584), 8192 x 5120 x 384 108 and 148 (2560), 32768 x 7168 x 72 179 and
// 194 (7168), but 16384 x 2560 x 256 82 and 76 (2560); 8192 x 2048 x 512 66 and 59, 8192
// x 4096 x 256 66 and 66 (2048), 4096 x 7168 x 256 59 and 57 (1792), 8192 x 4096 x 128
// 43 and 39 (1024), but where the tiles leave a last round half empty 8192 x 1024 x
// 1024 55 and 65 (1024) and 2000 x 6144 x 300 41 and 49 (768).  With BF16 weights, whose
// loads take more of the time than the products, 8192 x 7168 x 256 takes 58 and 56.
bool forward_pairs(const mega_moe_router_logits_args& a) {
    if (a.num_experts <= 64 || a.weight_type != MEGA_MOE_F32) return false;
    return a.hidden / split_for(forward_tiles(a), a.hidden, 256).n > 2048;
}

Plan forward_plan(const mega_moe_router_logits_args& a) {
    const int64_t T = a.num_tokens, E = a.num_experts, H = a.hidden;
    Plan p{};
    if (is_small(a, small_tile(a))) return p;
    // two workgroups to a compute unit, or one
    const bool two = E <= 32 ? a.weight_type == MEGA_MOE_BF16 : E <= 64 || forward_pairs(a);
    p.split = split_for(forward_tiles(a), H, two ? 512 : 256);
    p.total = p.split.n > 1 ? p.split.n * T * E * 4 : 0;
    return p;
}

Plan backward_plan(const mega_moe_router_logits_args& a) {
    const int64_t T = a.num_tokens, E = a.num_experts, H = a.hidden;
    Plan p{};
    p.split = split_for(tiles(E, 64) * tiles(H, 128), T, 256);     // few: they are joined again
    p.parts = T * padded(E) * 4;
    p.total = p.parts + (p.split.n > 1 ? p.split.n * E * H * 4 : 0);
    return p;
}

uint8_t* at(const mega_moe_router_logits_args& a, int64_t offset) { return static_cast<uint8_t*>(a.workspace) + offset; }

void launch_join(const float* parts, float* out, int64_t M, int64_t N, int64_t stride, int splits, hipStream_t stream) {
    const int64_t blocks = tiles(M * N, 1024);
    hipLaunchKernelGGL(moe_router_product_join, dim3((unsigned)(blocks > 65536 ? 65536 : blocks)), dim3(256), 0, stream,
                       parts, out, M, N, stride, splits);
}

// The forward product's kinds.  A float32 w is split where its fragments are
// read, so the fewer waves share columns, the less is split: with a wave's 32
// columns its own (1 x 4 waves) 8192 x 7168 x 256 takes 102 us and 512 x 7168 x
// 256 22, with planes of w in the workspace 112 and 27, and with 4 x 2 waves that
// split 155 and 26.
struct Bf16Forward {
    template <int BN, int STAGES, int WM, int WN>
    using Of = Kind<Lay::k_major, 1, Lay::k_major, 1, 128, BN, STAGES, false, WM, WN>;
    using Few = Of<32, 2, 4, 1>;
    using Some = Of<64, 2, 4, 1>;
    using Many = Of<128, 4, 4, 2>;
    using ManyPairs = Many;
};
struct F32Forward {
    template <int BN, int STAGES, int WM, int WN>
    using Of = Kind<Lay::k_major, 1, Lay::k_float, 3, 128, BN, STAGES, false, WM, WN>;
    using Few = Of<32, 4, 4, 1>;
    using Some = Of<64, 2, 2, 2>;
    // A workgroup to a compute unit, with a step in flight; and two of them that
    // hide each other's loads.
    using Many = Of<128, 2, 1, 4>;
    using ManyPairs = Of<128, 1, 1, 4>;
};

template <typename K>
void launch_product(const mega_moe_router_logits_args& a, hipStream_t stream) {
    const Plan p = forward_plan(a);
    const int64_t T = a.num_tokens, H = a.hidden, E = a.num_experts;
    float* parts = reinterpret_cast<float*>(at(a, p.parts));
    const Result out{T, E, p.split.n > 1 ? parts : a.logits, a.logits_stride, nullptr, nullptr, 0};
    const Product x{Operand{a.x, a.x_stride, T, H}, Operand{a.w, H, E, H}, out, p.split.k, p.split.n};
    hipLaunchKernelGGL((moe_router_product<K>), dim3((unsigned)(tiles(T, K::BM) * tiles(E, K::BN) * p.split.n)),
                       dim3(K::THREADS), 0, stream, x);
    if (p.split.n > 1) launch_join(parts, a.logits, T, E, a.logits_stride, p.split.n, stream);
}

template <typename F>
void launch_forward(const mega_moe_router_logits_args& a, hipStream_t stream) {
    if (a.num_experts <= 32) launch_product<typename F::Few>(a, stream);
    else if (a.num_experts <= 64) launch_product<typename F::Some>(a, stream);
    else if (forward_pairs(a)) launch_product<typename F::ManyPairs>(a, stream);
    else launch_product<typename F::Many>(a, stream);
}

// The gradients' kinds, with steps in LDS as they are launched.  In dx, which is
// rounded to BF16, two terms of dlogits do for BF16 weights: the 2^-17 that they leave
// shows only where the sum over the experts is some 256 times smaller than its terms,
// and rows of w of 8 bits hardly differ by so little (4096 x 4096 x 64 25 us, 26 with
// three terms; 8192 x 7168 x 256 181 and 198).  Float32 rows may: with what is 256 times
// their differences in common, and dlogits that add up to 0, as a softmax's do, two
// terms of both are half a step of BF16 (4096 x 4096 x 64 30 us and, with three, 33;
// 8192 x 7168 x 256 237 and 300).
struct Bf16Gradients {
    template <int S>
    using W = Kind<Lay::row_float, 3, Lay::row_major, 1, 64, 128, S, false>;
    template <int S>
    using X = Kind<Lay::k_float, 2, Lay::row_major, 1, 64, 128, S, true>;
};
struct F32Gradients {
    template <int S>
    using W = Bf16Gradients::W<S>;
    template <int S>
    using X = Kind<Lay::k_float, 3, Lay::row_float, 3, 64, 128, S, true>;
};

// Workgroups that a compute unit's 160 kB of LDS hold.
template <typename KW, typename KX>
constexpr unsigned to_a_unit() {
    return 163840u / ((KW::LDS > KX::LDS ? KW::LDS : KX::LDS) * 16u);
}

// One step in LDS or two.  Two, with which a workgroup keeps a step's loads in flight
// while it multiplies, where each has a place on the 256 compute units at once: two to
// a unit with BF16 weights (64 kB), one with float32 weights (96 kB).  More of them
// hide each other's loads, and with one step four and three to a unit fit.  One and
// two steps, us (workgroups), BF16 weights: 3383 x 640 x 216 21 and 19 (425), 768 x
// 3584 x 96 17 and 15 (448), 4096 x 2048 x 128 24 and 25 (1280), 4096 x 4096 x 64 25
// and 29 (2304), but 4096 x 896 x 64 17.7 and 16.9 (560); float32: 64 x 7168 x 256 13.2
// and 15.8 (280), 3383 x 640 x 216 24 and 29 (425), 768 x 3584 x 96 17 and 20 (448),
// 4096 x 4096 x 64 33 and 53 (2304), but 640 x 4096 x 64 14.6 and 13.8 (384) and 256 x
// 2048 x 128 8.6 and 8.3 (96).
template <typename G>
void launch_gradients(const Product& w, unsigned w_blocks, const Product& x, unsigned x_blocks, hipStream_t stream) {
    const auto go = [&](auto stages) {
        constexpr int S = decltype(stages)::value;
        hipLaunchKernelGGL((moe_router_gradients<typename G::template W<S>, typename G::template X<S>>),
                           dim3(w_blocks + x_blocks), dim3(256), 0, stream, w, w_blocks, x);
    };
    constexpr unsigned PLACES = 256 * to_a_unit<typename G::template W<2>, typename G::template X<2>>();
    if (w_blocks + x_blocks <= PLACES) go(std::integral_constant<int, 2>{});
    else go(std::integral_constant<int, 1>{});
}

}  // namespace

int64_t router_logits_workspace(const mega_moe_router_logits_args& a) {
    const int64_t f = forward_plan(a).total, b = backward_plan(a).total;
    return f > b ? f : b;
}

void launch_router_logits(const mega_moe_router_logits_args& a, hipStream_t stream) {
    const bool f = a.weight_type == MEGA_MOE_F32;
    const SmallTile s = small_tile(a);
    if (!is_small(a, s)) {
        if (f) launch_forward<F32Forward>(a, stream);
        else launch_forward<Bf16Forward>(a, stream);
        return;
    }
    const dim3 grid((unsigned)(tiles(a.num_tokens, s.t) * tiles(a.num_experts, s.e)));
    if (f) hipLaunchKernelGGL((moe_router_logits<true>), grid, dim3(1024), 0, stream, a, s.t, s.e);
    else hipLaunchKernelGGL((moe_router_logits<false>), grid, dim3(1024), 0, stream, a, s.t, s.e);
}

void launch_router_logits_backward(const mega_moe_router_logits_args& a, hipStream_t stream) {
    const int64_t T = a.num_tokens, H = a.hidden, E = a.num_experts, Ep = padded(E);
    const Plan p = backward_plan(a);
    const bool f = a.weight_type == MEGA_MOE_F32;
    // dlogits as it is where its rows are whole aligned chunks, and a tile of it
    // within 32-bit offsets
    const float* d = a.dlogits;
    int64_t d_stride = a.dlogits_stride;
    if (T > 0 && (E % 4 || d_stride % 4 || (uintptr_t)d % 16 || d_stride > MAX_TILE_STRIDE)) {
        float* to = reinterpret_cast<float*>(at(a, 0));
        const int64_t blocks = tiles(T * Ep / 4, 256);
        hipLaunchKernelGGL(moe_router_pad, dim3((unsigned)(blocks > 65536 ? 65536 : blocks)), dim3(256), 0, stream, d,
                           d_stride, T, (int)E, to, (int)Ep);
        d = to;
        d_stride = Ep;
    }
    const Product x{Operand{d, d_stride, T, Ep}, Operand{a.w, H, H, E},
                    Result{T, H, nullptr, a.dx_stride, a.dx, a.dx_add, a.dx_add_stride}, (Ep + 63) / 64 * 64, 1};
    float* parts = reinterpret_cast<float*>(at(a, p.parts));
    const Product w{Operand{d, d_stride, Ep, T}, Operand{a.x, a.x_stride, H, T},
                    Result{E, H, p.split.n > 1 ? parts : a.dw, H, nullptr, nullptr, 0}, p.split.k, p.split.n};
    const unsigned w_blocks = a.dw ? (unsigned)(tiles(E, 64) * tiles(H, 128) * p.split.n) : 0;
    const unsigned x_blocks = a.dx ? (unsigned)(tiles(T, 64) * tiles(H, 128)) : 0;
    if (f) launch_gradients<F32Gradients>(w, w_blocks, x, x_blocks, stream);
    else launch_gradients<Bf16Gradients>(w, w_blocks, x, x_blocks, stream);
    if (a.dw && p.split.n > 1) launch_join(parts, a.dw, E, H, H, p.split.n, stream);
}

}  // namespace mega_moe
