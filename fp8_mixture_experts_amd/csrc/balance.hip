// Per-expert route counts and the router's losses.
#include <hip/hip_runtime.h>

#include "moe_args.h"
#include "router.h"
#include "router_row.h"

namespace mega_moe {

// Workspace, for B sequences in S parts each: [B][S][E] floats (sums of p),
// [B][S][E] ints (counts), [B][S] floats (sums of lse^2), [B][S] ints (tokens),
// then [B] floats each: a sequence's balance term, its sum of lse^2.
struct BalanceWs {
    float* p;
    int32_t* count;
    float* z;
    int32_t* n;
    float* seq_loss;
    float* seq_z;
};

__host__ __device__ inline size_t balance_layout(int64_t B, int64_t S, int64_t E, char* base, BalanceWs& w) {
    size_t o = 0;
    const auto take = [&](size_t n) {
        char* p = base + o;
        o += (n + 15) / 16 * 16;
        return p;
    };
    w.p = (float*)take((size_t)(B * S * E) * 4);
    w.count = (int32_t*)take((size_t)(B * S * E) * 4);
    w.z = (float*)take((size_t)(B * S) * 4);
    w.n = (int32_t*)take((size_t)(B * S) * 4);
    w.seq_loss = (float*)take((size_t)B * 4);
    w.seq_z = (float*)take((size_t)B * 4);
    return o;
}

constexpr int BALANCE_ROWS = 32;      // tokens per part, about

__device__ __forceinline__ void sequence_span(const mega_moe_balance_loss_args& a, int b, int& lo, int& hi) {
    lo = 0;
    hi = a.num_tokens;
    if (a.cu_seqlens) {
        lo = min(max(a.cu_seqlens[b], 0), a.num_tokens);
        hi = min(max(a.cu_seqlens[b + 1], lo), a.num_tokens);
    }
}

// One part of one sequence per workgroup: a wave per token, its lanes keeping
// the sums of their experts; counts meet in LDS.
template <int NI>
__global__ void __launch_bounds__(256)
moe_balance_part(mega_moe_balance_loss_args a, BalanceWs ws, int S) {
    __shared__ int count[MAX_EXPERTS];
    __shared__ float sums[4][NI * 64];
    __shared__ float zs[4];
    __shared__ int ns[4];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int E = a.num_experts, k = a.num_topk;
    const int b = blockIdx.x / S, part = blockIdx.x - b * S;
    int lo, hi;
    sequence_span(a, b, lo, hi);
    const int64_t len = hi - lo;
    const int first = lo + (int)(len * part / S), last = lo + (int)(len * (part + 1) / S);
    for (int e = tid; e < E; e += 256) count[e] = 0;
    __syncthreads();
    float acc[NI], z = 0.0f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] = 0.0f;
    for (int t = first + wave; t < last; t += 4) {
        if (a.token_mask && a.token_mask[t] == 0) continue;
        ++n;
        float l[NI], ex[NI], top, sum;
        load_row<NI>(a.logits, a.logits_type, (size_t)t * a.logits_stride, E, l);
        row_exp(l, ex, top, sum);
        const float lse = row_lse(top, sum);
        z += lse * lse;
        if (a.score == MEGA_MOE_SCORE_SIGMOID) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                ex[i] = sigmoid(l[i]);
                s += ex[i];
            }
            sum = wave_sum(s);
        }
        const float inv = sum > 0.0f ? 1.0f / sum : sum;
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[i] += ex[i] * inv;
        for (int j = lane; j < k; j += 64) {
            const int e = a.topk_idx[(size_t)t * k + j];
            if (e >= 0 && e < E) atomicAdd(&count[e], 1);
        }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) sums[wave][i * 64 + lane] = acc[i];
    if (lane == 0) {
        zs[wave] = z;
        ns[wave] = n;
    }
    __syncthreads();
    for (int e = tid; e < E; e += 256) {
        ws.p[(size_t)blockIdx.x * E + e] = (sums[0][e] + sums[1][e]) + (sums[2][e] + sums[3][e]);
        ws.count[(size_t)blockIdx.x * E + e] = count[e];
    }
    if (tid == 0) {
        ws.z[blockIdx.x] = (zs[0] + zs[1]) + (zs[2] + zs[3]);
        ws.n[blockIdx.x] = ns[0] + ns[1] + ns[2] + ns[3];
    }
}

// One sequence per workgroup: its parts added up in order.
__global__ void __launch_bounds__(256)
moe_balance_sequence(mega_moe_balance_loss_args a, BalanceWs ws, int S) {
    __shared__ float part[16][1];
    const int b = blockIdx.x, tid = threadIdx.x, E = a.num_experts;
    int n = 0;
    float z = 0.0f;
    for (int s = 0; s < S; ++s) {
        n += ws.n[(size_t)b * S + s];
        z += ws.z[(size_t)b * S + s];
    }
    const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
    float dot[1] = {0.0f};
    for (int e = tid; e < E; e += 256) {
        float p = 0.0f;
        int c = 0;
        for (int s = 0; s < S; ++s) {
            p += ws.p[((size_t)b * S + s) * E + e];
            c += ws.count[((size_t)b * S + s) * E + e];
        }
        p *= inv;
        a.counts[(size_t)b * E + e] = c;
        if (a.probs) a.probs[(size_t)b * E + e] = p;
        dot[0] += (float)c * p;
    }
    block_sum(dot, part);
    if (tid == 0) {
        ws.seq_loss[b] = dot[0] * ((float)E / (float)a.num_topk) * inv;
        ws.seq_z[b] = z;
        a.tokens[b] = n;
    }
}

// The losses of all sequences.
__global__ void __launch_bounds__(256)
moe_balance_total(mega_moe_balance_loss_args a, BalanceWs ws, int B) {
    __shared__ float part[16][2];
    __shared__ int n_all, live_all;
    if (threadIdx.x == 0) n_all = live_all = 0;
    __syncthreads();
    float v[2] = {0.0f, 0.0f};
    int n = 0, live = 0;
    for (int b = threadIdx.x; b < B; b += 256) {
        v[0] += ws.seq_loss[b];
        v[1] += ws.seq_z[b];
        n += a.tokens[b];
        live += a.tokens[b] > 0;
    }
    atomicAdd(&n_all, n);
    atomicAdd(&live_all, live);
    block_sum(v, part);
    if (threadIdx.x == 0) {
        a.loss[0] = live_all ? a.balance_coeff * v[0] / (float)live_all : 0.0f;
        a.loss[1] = n_all ? a.z_coeff * v[1] / (float)n_all : 0.0f;
        a.tokens[B] = n_all;
        a.tokens[B + 1] = live_all;
    }
}

namespace {
int sequences(const mega_moe_balance_loss_args& a) { return a.cu_seqlens ? a.num_sequences : 1; }
// Parts per sequence: the host knows the sequences' average length only.
int parts(const mega_moe_balance_loss_args& a) {
    const int64_t B = sequences(a);
    const int64_t per = ((int64_t)a.num_tokens + B - 1) / B;
    const int64_t s = (per + BALANCE_ROWS - 1) / BALANCE_ROWS;
    return (int)(s < 1 ? 1 : s > 256 ? 256 : s);
}
}  // namespace

int64_t balance_loss_workspace(const mega_moe_balance_loss_args& a) {
    BalanceWs w;
    return (int64_t)balance_layout(sequences(a), parts(a), a.num_experts, nullptr, w);
}

void launch_balance_loss(const mega_moe_balance_loss_args& a, hipStream_t stream) {
    const int B = sequences(a), S = parts(a), E = a.num_experts;
    BalanceWs w;
    balance_layout(B, S, E, static_cast<char*>(a.workspace), w);
    const dim3 grid((unsigned)(B * S)), block(256);
    if (E <= 64) hipLaunchKernelGGL((moe_balance_part<1>), grid, block, 0, stream, a, w, S);
    else if (E <= 128) hipLaunchKernelGGL((moe_balance_part<2>), grid, block, 0, stream, a, w, S);
    else if (E <= 256) hipLaunchKernelGGL((moe_balance_part<4>), grid, block, 0, stream, a, w, S);
    else if (E <= 512) hipLaunchKernelGGL((moe_balance_part<8>), grid, block, 0, stream, a, w, S);
    else hipLaunchKernelGGL((moe_balance_part<16>), grid, block, 0, stream, a, w, S);
    hipLaunchKernelGGL(moe_balance_sequence, dim3((unsigned)B), block, 0, stream, a, w, S);
    hipLaunchKernelGGL(moe_balance_total, dim3(1), block, 0, stream, a, w, B);
}

}  // namespace mega_moe
