// The router's product, logits = x . w^T, and its gradients.
#include <hip/hip_runtime.h>

#include "block_util.h"
#include "router_logits.h"

namespace mega_moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Eight finite floats as the sum of P BF16 vectors.  Each term but the last is
// the leading eight significant bits of what is left (cut off, so it never
// overflows); with P = 3 the last holds the remaining eight bits, so the sum
// is exact, with P = 2 it is rounded to nearest: off by 2^-16 of the value.
template <int P>
__device__ __forceinline__ void split_bf16(const float (&v)[8], u32x4_t (&p)[3]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float r[2] = {v[2 * i], v[2 * i + 1]};
#pragma unroll
        for (int q = 0; q + 1 < P; ++q) {
            const uint32_t a = __float_as_uint(r[0]), b = __float_as_uint(r[1]);
            p[q][i] = __builtin_amdgcn_perm(b, a, 0x07060302u);      // the upper halves
            r[0] -= __uint_as_float(a & 0xffff0000u);
            r[1] -= __uint_as_float(b & 0xffff0000u);
        }
        p[P - 1][i] = P == 3 ? __builtin_amdgcn_perm(__float_as_uint(r[1]), __float_as_uint(r[0]), 0x07060302u)
                             : bf16_pair(r[0], r[1]);
    }
}

// Small batches.  A tile of up to 16 tokens x 16 experts per workgroup; its 16
// waves take the K steps of 32 in turn, straight from memory, and their sums
// meet in LDS.  What bounds it is how fast one compute unit takes in its rows
// (about 40 GB/s, whatever the others do), so the tile is the one that leaves
// the fewest bytes to each (small_tile below) and fills the rest of the matrix
// instruction with zeros, and each wave has the loads of STEPS steps in flight
// (H = 7168: its 14 steps in two rounds).  128 x 7168 x 32: 14 us with whole
// tiles on 16 compute units, 6.5 us with 4 x 4 on 256.
template <bool WF32>
__global__ void __launch_bounds__(1024)
moe_router_logits(mega_moe_router_logits_args a, int tile_t, int tile_e) {
    constexpr int STEPS = 7;
    __shared__ float part[16][16][17];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, kq = (lane >> 4) * 8;
    const int H = a.hidden, E = a.num_experts;
    const int e_tiles = (E + tile_e - 1) / tile_e;
    const int e0 = (int)(blockIdx.x % e_tiles) * tile_e;
    const int t0 = (int)(blockIdx.x / e_tiles) * tile_t;
    const bool has_t = r < tile_t && t0 + r < a.num_tokens, has_e = r < tile_e && e0 + r < E;
    const uint16_t* x = a.x + (int64_t)(t0 + r) * a.x_stride;
    const size_t w_row = (size_t)(e0 + r) * H;
    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = wave * 32; k0 < H; k0 += 512 * STEPS) {
        u32x4_t xv[STEPS], wv[STEPS][WF32 ? 2 : 1];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int k = k0 + s * 512 + kq;
            const u32x4_t none = {0u, 0u, 0u, 0u};
            xv[s] = none;
#pragma unroll
            for (int i = 0; i < (WF32 ? 2 : 1); ++i) wv[s][i] = none;
            if (has_t && k < H) xv[s] = *reinterpret_cast<const u32x4_t*>(x + k);
            if (has_e && k < H) {
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
    for (int i = 0; i < 4; ++i) part[wave][r][(lane >> 4) * 4 + i] = acc[i];
    __syncthreads();
    if (threadIdx.x >= 256) return;
    const int to = threadIdx.x >> 4, eo = threadIdx.x & 15;
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < 16; ++w) s += part[w][to][eo];
    if (to < tile_t && eo < tile_e && t0 + to < a.num_tokens && e0 + eo < E)
        a.logits[(int64_t)(t0 + to) * a.logits_stride + e0 + eo] = s;
}

// ---------------------------------------------------------------------------
// Tiles through LDS, for batches of tokens and for the gradients.
// C[m, n] = sum over k of A[m, k] B[n, k] on 32 x 32 x 16 BF16 matrix
// instructions.  A workgroup of four waves computes BM x BN; every
// K step of 64 goes through registers into LDS, as one to three BF16 planes
// per operand (a float32 operand is split there), and the planes' products add
// into the same accumulators, the small ones first.
//
// LDS: a plane is [rows][64] BF16, 128 bytes a row in eight 16-byte chunks;
// chunk c of row r lies at c ^ (r & 7), so that the 16-byte reads of eight
// rows at one k spread over all banks.
// ---------------------------------------------------------------------------

// How an operand lies in memory: K contiguous ([rows][K], a chunk of eight k
// is one or two 16-byte loads) or rows contiguous ([K][rows], eight k of two
// rows are eight loads that the registers turn around).
enum class Lay { k_major, row_major };

struct Operand {
    const void* p;
    int64_t stride;        // elements from one row (k_major) or k (row_major) to the next
    int64_t rows, k;       // valid extents
};

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4a_t __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2a_t __attribute__((ext_vector_type(2), aligned(4)));

// One operand's share of a K step in this thread's registers.
template <bool F32, Lay L, int R>
struct Staged {
    // k_major: R / 32 chunks; row_major: R / 64 units of 8 k x 2 rows
    static constexpr int N = L == Lay::k_major ? R / 32 : R / 64;
    static constexpr int W = L == Lay::k_major ? (F32 ? 8 : 4) : (F32 ? 16 : 8);
    uint32_t v[N][W];

    __device__ __forceinline__ void load(const Operand& o, int64_t row0, int64_t k0, int64_t k_end) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int id = i * 256 + tid;
#pragma unroll
            for (int j = 0; j < W; ++j) v[i][j] = 0u;
            if constexpr (L == Lay::k_major) {
                const int64_t r = row0 + (id >> 3), k = k0 + (id & 7) * 8;
                if (r >= o.rows || k >= k_end) continue;
                if constexpr (F32) {
                    const uint32_t* q = static_cast<const uint32_t*>(o.p) + r * o.stride + k;
                    if (k + 8 <= k_end) {
                        const u32x4a_t a = *reinterpret_cast<const u32x4a_t*>(q);
                        const u32x4a_t b = *reinterpret_cast<const u32x4a_t*>(q + 4);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[i][j] = a[j], v[i][4 + j] = b[j];
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (k + j < k_end) v[i][j] = q[j];
                    }
                } else {
                    // BF16 rows are whole chunks of eight
                    const u32x4_t a = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(o.p) + r * o.stride + k);
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = a[j];
                }
            } else {
                const int64_t r = row0 + (id % (R / 2)) * 2, k = k0 + (id / (R / 2)) * 8;
                if (r >= o.rows) continue;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (k + j >= k_end) break;
                    if constexpr (F32) {
                        const uint32_t* q = static_cast<const uint32_t*>(o.p) + (k + j) * o.stride + r;
                        if (r + 1 < o.rows) {
                            const u32x2a_t a = *reinterpret_cast<const u32x2a_t*>(q);
                            v[i][2 * j] = a[0];
                            v[i][2 * j + 1] = a[1];
                        } else {
                            v[i][2 * j] = q[0];
                        }
                    } else {
                        // the rows come in eights
                        v[i][j] = *reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(o.p) + (k + j) * o.stride + r);
                    }
                }
            }
        }
    }

    // Writes the chunks as P planes (1: BF16 as it is).
    template <int P>
    __device__ __forceinline__ void store(u32x4_t* lds) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int id = i * 256 + tid;
#pragma unroll
            for (int h = 0; h < (L == Lay::k_major ? 1 : 2); ++h) {
                const int r = L == Lay::k_major ? id >> 3 : (id % (R / 2)) * 2 + h;
                const int c = L == Lay::k_major ? id & 7 : id / (R / 2);
                u32x4_t* at = lds + r * 8 + (c ^ (r & 7));
                if constexpr (F32) {
                    float x[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(L == Lay::k_major ? v[i][j] : v[i][2 * j + h]);
                    u32x4_t p[3];
                    split_bf16<P>(x, p);
#pragma unroll
                    for (int q = 0; q < P; ++q) at[q * R * 8] = p[q];
                } else if constexpr (L == Lay::k_major) {
                    *at = u32x4_t{v[i][0], v[i][1], v[i][2], v[i][3]};
                } else {
                    u32x4_t p;
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        p[j] = h == 0 ? (v[i][2 * j] & 0xffffu) | (v[i][2 * j + 1] << 16)
                                      : (v[i][2 * j] >> 16) | (v[i][2 * j + 1] & 0xffff0000u);
                    *at = p;
                }
            }
        }
    }
};

// Where a product goes: float32 rows (the result, or one split's part of it in
// the workspace, [split][M][N]), or BF16 rows with something added.
struct Result {
    float* f32;
    int64_t stride;
    uint16_t* bf16;
    const uint16_t* add;
    int64_t add_stride;
};

template <bool AF32, Lay AL, int PA, bool BF32, Lay BL, int PB, int BM, int BN, bool OUT_BF16>
__global__ void __launch_bounds__(256)
moe_router_product(Operand A, Operand Bo, Result out, int64_t k_split, int splits) {
    // BF16 results go out through LDS, as rows of floats
    constexpr int PITCH = BN + 4;
    constexpr int STAGE = (PA * BM + PB * BN) * 8, OUT = OUT_BF16 ? BM * PITCH / 4 : 0;
    __shared__ u32x4_t lds[STAGE > OUT ? STAGE : OUT];
    u32x4_t* la = lds;
    u32x4_t* lb = lds + PA * BM * 8;
    // waves over the tile: 2 x 2 where it is wide, else all along M
    constexpr int WN = BN >= 128 || BM < 128 ? 2 : 1, WM = 4 / WN;
    constexpr int TM = BM / WM / 32, TN = BN / WN / 32;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wm = wave / WN * (TM * 32), wn = wave % WN * (TN * 32);
    const int n_tiles = (int)((Bo.rows + BN - 1) / BN);
    const int split = blockIdx.x % splits;
    const int64_t tile = blockIdx.x / splits;
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

    Staged<AF32, AL, BM> sa;
    Staged<BF32, BL, BN> sb;
    if (k_first < k_end) {
        sa.load(A, m0, k_first, k_end);
        sb.load(Bo, n0, k_first, k_end);
    }
    for (int64_t k0 = k_first; k0 < k_end; k0 += 64) {
        sa.template store<PA>(la);
        sb.template store<PB>(lb);
        __syncthreads();
        if (k0 + 64 < k_end) {
            sa.load(A, m0, k0 + 64, k_end);
            sb.load(Bo, n0, k0 + 64, k_end);
        }
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            const int c = kk * 2 + (lane >> 5), r = lane & 31;
            bf16x8_t fa[PA][TM], fb[PB][TN];
#pragma unroll
            for (int p = 0; p < PA; ++p)
#pragma unroll
                for (int i = 0; i < TM; ++i)
                    fa[p][i] = __builtin_bit_cast(bf16x8_t, la[(p * BM + wm + i * 32 + r) * 8 + (c ^ (r & 7))]);
#pragma unroll
            for (int p = 0; p < PB; ++p)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    fb[p][j] = __builtin_bit_cast(bf16x8_t, lb[(p * BN + wn + j * 32 + r) * 8 + (c ^ (r & 7))]);
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
        }
        __syncthreads();
    }

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
        for (int i = 0; i < BM * BN / 8 / 256; ++i) {
            const int id = i * 256 + (int)threadIdx.x;
            const int r = id / (BN / 8), c = id % (BN / 8) * 8;
            const int64_t m = m0 + r, n = n0 + c;
            if (m >= A.rows || n >= Bo.rows) continue;      // the rows come in eights
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
            if (m >= A.rows) continue;
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int64_t n = n0 + wn + j * 32 + g * 8 + (lane >> 5) * 4;
                    if (n >= Bo.rows) continue;
                    float v[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = acc[i][j][g * 4 + q];
                    float* o = out.f32 + (splits > 1 ? split * A.rows * Bo.rows + m * Bo.rows : m * out.stride) + n;
                    if (n + 4 <= Bo.rows) {
                        u32x4a_t d;
#pragma unroll
                        for (int q = 0; q < 4; ++q) d[q] = __float_as_uint(v[q]);
                        *reinterpret_cast<u32x4a_t*>(o) = d;
                    } else {
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            if (n + q < Bo.rows) o[q] = v[q];
                    }
                }
        }
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

constexpr int64_t SMALL_TOKENS = 256;    // up to here the 16 x 16 tiles compute the logits

struct Split {
    int n;               // parts of K
    int64_t k;           // K of a part, whole steps of 64
};

// Parts of K for a product of `tiles` tiles: enough to give every compute unit
// two workgroups, each with four steps or more.
Split split_for(int64_t tiles, int64_t K) {
    int n = 1;
    while (n < 16 && tiles * n < 512 && K / (2 * n) >= 256) n *= 2;
    const int64_t steps = (K + 63) / 64;
    return Split{n, (steps + n - 1) / n * 64};
}

int columns(int64_t E) { return E <= 32 ? 32 : E <= 64 ? 64 : 128; }
int64_t tiles(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tile of a small batch: the fewest rows, by their bytes, for one compute
// unit of 256, in as many turns as the tiles take.
struct SmallTile {
    int t, e;
};
SmallTile small_tile(const mega_moe_router_logits_args& a) {
    const int w_bytes = a.weight_type == MEGA_MOE_F32 ? 4 : 2;
    SmallTile best{16, 16};
    int64_t least = INT64_MAX;
    for (int t = 16; t >= 1; t /= 2)
        for (int e = 16; e >= 1; e /= 2) {
            const int64_t turns = tiles(tiles(a.num_tokens, t) * tiles(a.num_experts, e), 256);
            const int64_t bytes = turns * (t * 2 + e * w_bytes);
            if (bytes < least) least = bytes, best = SmallTile{t, e};
        }
    return best;
}

Split forward_split(const mega_moe_router_logits_args& a) {
    return split_for(tiles(a.num_tokens, 128) * tiles(a.num_experts, columns(a.num_experts)), a.hidden);
}
Split dw_split(const mega_moe_router_logits_args& a) {
    return split_for(tiles(a.num_experts, 64) * tiles(a.hidden, 64), a.num_tokens);
}

void launch_join(const mega_moe_router_logits_args& a, float* out, int64_t M, int64_t N, int64_t stride, int splits,
                 hipStream_t stream) {
    const int64_t blocks = tiles(M * N, 1024);
    hipLaunchKernelGGL(moe_router_product_join, dim3((unsigned)(blocks > 65536 ? 65536 : blocks)), dim3(256), 0, stream,
                       static_cast<const float*>(a.workspace), out, M, N, stride, splits);
}

template <bool WF32, int BN>
void launch_logits(const mega_moe_router_logits_args& a, hipStream_t stream) {
    const Split s = forward_split(a);
    const int64_t T = a.num_tokens, H = a.hidden, E = a.num_experts;
    const Operand A{a.x, a.x_stride, T, H}, W{a.w, H, E, H};
    const Result out{s.n > 1 ? static_cast<float*>(a.workspace) : a.logits, a.logits_stride, nullptr, nullptr, 0};
    hipLaunchKernelGGL((moe_router_product<false, Lay::k_major, 1, WF32, Lay::k_major, WF32 ? 3 : 1, 128, BN, false>),
                       dim3((unsigned)(tiles(T, 128) * tiles(E, BN) * s.n)), dim3(256), 0, stream, A, W, out, s.k, s.n);
    if (s.n > 1) launch_join(a, a.logits, T, E, a.logits_stride, s.n, stream);
}

}  // namespace

int64_t router_logits_workspace(const mega_moe_router_logits_args& a) {
    const int64_t T = a.num_tokens, E = a.num_experts, H = a.hidden;
    const Split f = forward_split(a), d = dw_split(a);
    const int64_t forward = T > SMALL_TOKENS && f.n > 1 ? f.n * T * E * 4 : 0;
    const int64_t backward = d.n > 1 ? d.n * E * H * 4 : 0;
    return forward > backward ? forward : backward;
}

void launch_router_logits(const mega_moe_router_logits_args& a, hipStream_t stream) {
    const bool f = a.weight_type == MEGA_MOE_F32;
    if (a.num_tokens > SMALL_TOKENS) {
        const int bn = columns(a.num_experts);
        if (f) {
            if (bn == 32) launch_logits<true, 32>(a, stream);
            else if (bn == 64) launch_logits<true, 64>(a, stream);
            else launch_logits<true, 128>(a, stream);
        } else {
            if (bn == 32) launch_logits<false, 32>(a, stream);
            else if (bn == 64) launch_logits<false, 64>(a, stream);
            else launch_logits<false, 128>(a, stream);
        }
        return;
    }
    const SmallTile s = small_tile(a);
    const dim3 grid((unsigned)(tiles(a.num_tokens, s.t) * tiles(a.num_experts, s.e)));
    if (f) hipLaunchKernelGGL((moe_router_logits<true>), grid, dim3(1024), 0, stream, a, s.t, s.e);
    else hipLaunchKernelGGL((moe_router_logits<false>), grid, dim3(1024), 0, stream, a, s.t, s.e);
}

void launch_router_logits_backward(const mega_moe_router_logits_args& a, hipStream_t stream) {
    const int64_t T = a.num_tokens, H = a.hidden, E = a.num_experts;
    if (a.dx && T > 0) {
        const Operand D{a.dlogits, a.dlogits_stride, T, E}, W{a.w, H, H, E};
        const Result out{nullptr, a.dx_stride, a.dx, a.dx_add, a.dx_add_stride};
        const dim3 grid((unsigned)(tiles(T, 64) * tiles(H, 128)));
        if (a.weight_type == MEGA_MOE_F32)
            hipLaunchKernelGGL((moe_router_product<true, Lay::k_major, 2, true, Lay::row_major, 2, 64, 128, true>), grid,
                               dim3(256), 0, stream, D, W, out, (E + 63) / 64 * 64, 1);
        else
            hipLaunchKernelGGL((moe_router_product<true, Lay::k_major, 2, false, Lay::row_major, 1, 64, 128, true>), grid,
                               dim3(256), 0, stream, D, W, out, (E + 63) / 64 * 64, 1);
    }
    if (a.dw) {
        const Split s = dw_split(a);
        const Operand D{a.dlogits, a.dlogits_stride, E, T}, X{a.x, a.x_stride, H, T};
        const Result out{s.n > 1 ? static_cast<float*>(a.workspace) : a.dw, H, nullptr, nullptr, 0};
        hipLaunchKernelGGL((moe_router_product<true, Lay::row_major, 3, false, Lay::row_major, 1, 64, 64, false>),
                           dim3((unsigned)(tiles(E, 64) * tiles(H, 64) * s.n)), dim3(256), 0, stream, D, X, out, s.k, s.n);
        if (s.n > 1) launch_join(a, a.dw, E, H, H, s.n, stream);
    }
}

}  // namespace mega_moe
