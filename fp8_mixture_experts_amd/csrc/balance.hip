// Per-expert route counts and the router's losses, in two launches.
//
// moe_balance_part takes the tokens in chunks of 32, one per workgroup, and
// writes a record (sums of p and counts per expert, sum of lse^2, tokens) for
// every sequence that has tokens in the chunk: chunk c and sequence b have
// record c + b, which no other pair has, since both grow along the tokens; a
// sequence's records lie next to each other.  The lengths of the sequences,
// which the host does not know, thus never unbalance the work.
// moe_balance_finish adds up every sequence's records in order, 32 experts per
// workgroup; the workgroup that ends last adds up the losses.
//
// The logits are read once (8 MB at 8192 x 256: 2 us); what bounds it is the
// chain of a token's loads, exponentials and sums, and the two launches: 8.6 and
// 5.6 us there, with 13 sequences; 3.5 and 2.6 us at 576 x 32.  p is computed once
// for all the sequences that a chunk meets: computed for each of them in turn,
// 32768 x 256 with 64 sequences took a third longer than so (17.4 and 12.5 us).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "moe_args.h"
#include "router.h"
#include "router_row.h"

namespace mega_moe {

constexpr int CHUNK = 32;             // tokens per chunk
constexpr int SLICE = BALANCE_SLICE;

struct BalanceWs {
    float* p;             // [records][E]
    int32_t* count;       // [records][E]
    float* z;             // [records]
    int32_t* n;           // [records]
    float* seq_loss;      // [B][slices] a sequence's balance term
    float* seq_z;         // [B] its sum of lse^2
    uint32_t* done;       // workgroups of the second launch that have ended
};

__host__ __device__ inline int64_t balance_chunks(int64_t T) { return (T + CHUNK - 1) / CHUNK; }

__host__ __device__ inline size_t balance_layout(int64_t T, int64_t B, int64_t E, char* base, BalanceWs& w) {
    const int64_t records = balance_chunks(T) + B;
    size_t o = 0;
    const auto take = [&](size_t n) {
        char* p = base + o;
        o += (n + 15) / 16 * 16;
        return p;
    };
    w.p = (float*)take((size_t)(records * E) * 4);
    w.count = (int32_t*)take((size_t)(records * E) * 4);
    w.z = (float*)take((size_t)records * 4);
    w.n = (int32_t*)take((size_t)records * 4);
    w.seq_loss = (float*)take((size_t)(B * ((E + SLICE - 1) / SLICE)) * 4);
    w.seq_z = (float*)take((size_t)B * 4);
    w.done = (uint32_t*)take(4);
    return o;
}

// Sequence b's tokens, within [0, T) whatever cu_seqlens holds.
__device__ __forceinline__ void sequence_span(const mega_moe_balance_loss_args& a, int b, int& lo, int& hi) {
    lo = 0;
    hi = a.num_tokens;
    if (a.cu_seqlens) {
        lo = min(max(a.cu_seqlens[b], 0), a.num_tokens);
        hi = min(max(a.cu_seqlens[b + 1], lo), a.num_tokens);
    }
}

// A token's experts lie in LANES lanes; the groups of lanes take the tokens in
// turn, each lane keeping the sums of its experts.
constexpr int part_threads(int lanes) { return lanes == 32 ? 1024 : 512; }

template <int LANES, int NI>
__global__ void __launch_bounds__(part_threads(LANES))
moe_balance_part(mega_moe_balance_loss_args a, BalanceWs ws, int B) {
    constexpr int THREADS = part_threads(LANES), WAVES = THREADS / 64, GROUPS = THREADS / LANES;
    __shared__ int count[LANES * NI];
    __shared__ float sums[WAVES][LANES * NI];
    __shared__ float zs[WAVES];
    __shared__ int ns[WAVES];
    const int tid = threadIdx.x, lane = tid & (LANES - 1), group = tid / LANES, wave = tid >> 6;
    const int E = a.num_experts, k = a.num_topk;
    const int c0 = blockIdx.x * CHUNK, c1 = min(c0 + CHUNK, a.num_tokens);
    if (blockIdx.x == 0 && tid == 0) *ws.done = 0;
    // the ends of up to 64 sequences, in every wave's lanes: asked for first, so
    // that the look-up below waits for nothing that the logits do not wait for
    const bool in_lanes = a.cu_seqlens && B <= 64;
    int ends = 0x7fffffff, start = 0;
    if (in_lanes) {
        start = a.cu_seqlens[0];
        if ((tid & 63) < B) ends = a.cu_seqlens[(tid & 63) + 1];
    }
    constexpr int ROWS = CHUNK / GROUPS;         // tokens per group
    const bool sigmoids = a.score == MEGA_MOE_SCORE_SIGMOID;
    float l[ROWS][NI];
    int slot[ROWS];
    bool live[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int t = c0 + r * GROUPS + group;
        live[r] = t < c1 && (!a.token_mask || a.token_mask[t] != 0);
        slot[r] = t < c1 && lane < k ? a.topk_idx[(size_t)t * k + lane] : -1;
        if (t < c1) {
            load_row<NI, LANES>(a.logits, a.logits_type, (size_t)t * a.logits_stride, E, l[r]);
        } else {
#pragma unroll
            for (int i = 0; i < NI; ++i) l[r][i] = 0.0f;
        }
    }
    // the logits become p, once for all the sequences that the chunk meets
    float zr[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        float ex[NI], top, sum = 0.0f;
        zr[r] = 0.0f;
        if (!sigmoids || a.z_coeff != 0.0f) {
            row_exp<LANES>(l[r], ex, top, sum);
            const float lse = row_lse(top, sum);
            zr[r] = lse * lse;
        }
        if (sigmoids) {
            sum = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                ex[i] = sigmoid(l[r][i]);
                sum += ex[i];
            }
            sum = lanes_sum<LANES>(sum);
            if (sum < SMALL_SUM) row_exp<LANES>(l[r], ex, top, sum);
        }
        const float inv = sum > 0.0f ? 1.0f / sum : sum;
#pragma unroll
        for (int i = 0; i < NI; ++i) l[r][i] = ex[i] * inv;
    }
    int p = c0;
    while (p < c1) {
        int b, lo, hi;
        if (in_lanes) {
            // as many sequences end at p or before
            const int n = __builtin_popcountll(__builtin_amdgcn_ballot_w64(ends <= p));
            b = p < start || n >= B ? -1 : n;
            hi = __builtin_amdgcn_readlane(ends, b < 0 ? 0 : b);
        } else {
            b = sequence_of<64>(a.cu_seqlens, B, p);
            if (b >= 0) sequence_span(a, b, lo, hi);
            else start = a.cu_seqlens[0];
        }
        if (b < 0) {
            // before the first sequence, or behind the last
            if (p >= start) break;
            p = start;
            continue;
        }
        if (hi <= p) break;                      // cu_seqlens decreases
        const int end = min(hi, c1);
        for (int e = tid; e < LANES * NI; e += THREADS) count[e] = 0;
        __syncthreads();
        float acc[NI], z = 0.0f;
        int n = 0;
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int t = c0 + r * GROUPS + group;
            if (!live[r] || t < p || t >= end) continue;
            ++n;
            z += zr[r];
#pragma unroll
            for (int i = 0; i < NI; ++i) acc[i] += l[r][i];
            if (slot[r] >= 0 && slot[r] < E) atomicAdd(&count[slot[r]], 1);
            for (int j = lane + LANES; j < k; j += LANES) {
                const int e = a.topk_idx[(size_t)t * k + j];
                if (e >= 0 && e < E) atomicAdd(&count[e], 1);
            }
        }
        // the wave's groups of lanes, then the waves, in order
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            if constexpr (LANES <= 16) acc[i] += __shfl_xor(acc[i], 16, 64);
            if constexpr (LANES <= 32) acc[i] += __shfl_xor(acc[i], 32, 64);
            if ((tid & 63) < LANES) sums[wave][i * LANES + lane] = acc[i];
        }
        if constexpr (LANES <= 16) z += __shfl_xor(z, 16, 64), n += __shfl_xor(n, 16, 64);
        if constexpr (LANES <= 32) z += __shfl_xor(z, 32, 64), n += __shfl_xor(n, 32, 64);
        if ((tid & 63) == 0) {
            zs[wave] = z;
            ns[wave] = n;
        }
        __syncthreads();
        const size_t rec = (size_t)blockIdx.x + b;
        for (int e = tid; e < E; e += THREADS) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) s += sums[w][e];
            ws.p[rec * E + e] = s;
            ws.count[rec * E + e] = count[e];
        }
        if (tid == 0) {
            float zt = 0.0f;
            int nt = 0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                zt += zs[w];
                nt += ns[w];
            }
            ws.z[rec] = zt;
            ws.n[rec] = nt;
        }
        __syncthreads();
        p = end;
    }
}

// Workgroup (b, slice): GROUPS groups of 32 threads add up every GROUPS-th
// record of sequence b for 32 experts, and meet in LDS.
template <int GROUPS>
__global__ void __launch_bounds__(GROUPS * SLICE)
moe_balance_finish(mega_moe_balance_loss_args a, BalanceWs ws, int B) {
    __shared__ float sp[GROUPS][SLICE];
    __shared__ int sc[GROUPS][SLICE], n_part[16], live_part[16];
    __shared__ float z_part[16][1], loss_part[16][2];
    __shared__ bool last;
    const int tid = threadIdx.x, x = tid & (SLICE - 1), g = tid / SLICE, wave = tid >> 6;
    constexpr int WAVES = (GROUPS * SLICE + 63) / 64;
    const int E = a.num_experts, slices = (E + SLICE - 1) / SLICE;
    const int b = blockIdx.x / slices, slice = blockIdx.x - b * slices, e = slice * SLICE + x;
    int lo, hi;
    sequence_span(a, b, lo, hi);
    const size_t first = (size_t)(lo / CHUNK) + b;
    const int records = hi > lo ? (hi - 1) / CHUNK - lo / CHUNK + 1 : 0;
    float p = 0.0f, z[1] = {0.0f};
    int c = 0, n = 0;
    if (e < E) {
#pragma unroll 8
        for (int r = g; r < records; r += GROUPS) {
            p += ws.p[(first + r) * E + e];
            c += ws.count[(first + r) * E + e];
        }
    }
    for (int r = tid; r < records; r += GROUPS * SLICE) {
        n += ws.n[first + r];
        z[0] += ws.z[first + r];
    }
    sp[g][x] = p;
    sc[g][x] = c;
    n = (int)over_lanes<64>((uint32_t)n, [](uint32_t u, uint32_t v) { return u + v; });
    if ((tid & 63) == 0) n_part[wave] = n;
    block_sum(z, z_part);
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) n += n_part[w];
    const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
    if (tid < 64) {
        float dot = 0.0f;
        if (tid < SLICE && e < E) {
            p = 0.0f;
            c = 0;
#pragma unroll
            for (int q = 0; q < GROUPS; ++q) {
                p += sp[q][x];
                c += sc[q][x];
            }
            p *= inv;
            a.counts[(size_t)b * E + e] = c;
            if (a.probs) a.probs[(size_t)b * E + e] = p;
            dot = (float)c * p;
        }
        dot = wave_sum(dot);
        if (tid == 0 && gridDim.x == 1) {
            // nothing to wait for
            a.loss[0] = n > 0 ? a.balance_coeff * (dot * ((float)E / (float)a.num_topk) * inv) : 0.0f;
            a.loss[1] = n > 0 ? a.z_coeff * z[0] / (float)n : 0.0f;
            a.tokens[0] = a.tokens[1] = n;
            a.tokens[2] = n > 0;
            last = false;
        } else if (tid == 0) {
            // read by the last workgroup, from another die perhaps: past its L2
            __hip_atomic_store(ws.seq_loss + (size_t)b * slices + slice, dot * ((float)E / (float)a.num_topk) * inv,
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            if (slice == 0) {
                __hip_atomic_store(ws.seq_z + b, z[0], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                __hip_atomic_store(a.tokens + b, n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            }
            last = __hip_atomic_fetch_add(ws.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == gridDim.x - 1;
        }
    }
    __syncthreads();
    if (!last) return;
    float v[2] = {0.0f, 0.0f};
    int all = 0, live = 0;
    for (int64_t i = tid; i < (int64_t)B * slices; i += GROUPS * SLICE)
        v[0] += __hip_atomic_load(ws.seq_loss + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    for (int i = tid; i < B; i += GROUPS * SLICE) {
        v[1] += __hip_atomic_load(ws.seq_z + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        const int m = __hip_atomic_load(a.tokens + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        all += m;
        live += m > 0;
    }
    const auto add = [](uint32_t u, uint32_t w) { return u + w; };
    all = (int)over_lanes<64>((uint32_t)all, add);
    live = (int)over_lanes<64>((uint32_t)live, add);
    if ((tid & 63) == 0) {
        n_part[wave] = all;
        live_part[wave] = live;
    }
    block_sum(v, loss_part);
    __syncthreads();
    if (tid == 0) {
        all = live = 0;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            all += n_part[w];
            live += live_part[w];
        }
        a.loss[0] = live ? a.balance_coeff * v[0] / (float)live : 0.0f;
        a.loss[1] = all ? a.z_coeff * v[1] / (float)all : 0.0f;
        a.tokens[B] = all;
        a.tokens[B + 1] = live;
    }
}

namespace {
int sequences(const mega_moe_balance_loss_args& a) { return a.cu_seqlens ? a.num_sequences : 1; }
}  // namespace

int64_t balance_loss_workspace(const mega_moe_balance_loss_args& a) {
    BalanceWs w;
    return (int64_t)balance_layout(a.num_tokens, sequences(a), a.num_experts, nullptr, w);
}

void launch_balance_loss(const mega_moe_balance_loss_args& a, hipStream_t stream) {
    const int B = sequences(a), E = a.num_experts;
    BalanceWs w;
    balance_layout(a.num_tokens, B, E, static_cast<char*>(a.workspace), w);
    const int64_t chunks = balance_chunks(a.num_tokens);
    const dim3 grid((unsigned)(chunks > 0 ? chunks : 1));
    const auto part = [&](auto lanes, auto ni) {
        constexpr int L = decltype(lanes)::value, NI = decltype(ni)::value;
        hipLaunchKernelGGL((moe_balance_part<L, NI>), grid, dim3(part_threads(L)), 0, stream, a, w, B);
    };
    using std::integral_constant;
    if (E <= 16) part(integral_constant<int, 16>{}, integral_constant<int, 1>{});
    else if (E <= 32) part(integral_constant<int, 16>{}, integral_constant<int, 2>{});
    else if (E <= 64) part(integral_constant<int, 16>{}, integral_constant<int, 4>{});
    else if (E <= 128) part(integral_constant<int, 32>{}, integral_constant<int, 4>{});
    else if (E <= 256) part(integral_constant<int, 32>{}, integral_constant<int, 8>{});
    else if (E <= 512) part(integral_constant<int, 64>{}, integral_constant<int, 8>{});
    else part(integral_constant<int, 64>{}, integral_constant<int, 16>{});
    const dim3 finish((unsigned)balance_finish_groups(B, E));
    if (chunks / B >= 16) hipLaunchKernelGGL((moe_balance_finish<32>), finish, dim3(1024), 0, stream, a, w, B);
    else hipLaunchKernelGGL((moe_balance_finish<8>), finish, dim3(256), 0, stream, a, w, B);
}

}  // namespace mega_moe
