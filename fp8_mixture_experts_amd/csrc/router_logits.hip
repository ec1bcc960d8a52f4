// The router's product, logits = x . w^T, and its gradients.
#include <hip/hip_runtime.h>

#include "block_util.h"
#include "router_logits.h"

namespace mega_moe {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// Eight floats as the sum of three BF16 vectors: each term is the leading
// eight significant bits of what is left, so the sum is exact (24 bits).  An
// infinity or NaN goes into the first term alone.
__device__ __forceinline__ void split3(const float (&v)[8], bf16x8_t& hi, bf16x8_t& mid, bf16x8_t& lo) {
    u32x4_t h, m, l;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint32_t a[2], b[2], c[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float x = v[2 * i + j];
            a[j] = __float_as_uint(x) & 0xffff0000u;
            const float r1 = (a[j] & 0x7f800000u) == 0x7f800000u ? 0.0f : x - __uint_as_float(a[j]);
            b[j] = __float_as_uint(r1) & 0xffff0000u;
            c[j] = __float_as_uint(r1 - __uint_as_float(b[j]));
            if ((__float_as_uint(x) & 0x7fffffffu) > 0x7f800000u) a[j] = 0x7fc00000u;
        }
        h[i] = (a[0] >> 16) | a[1];
        m[i] = (b[0] >> 16) | b[1];
        l[i] = (c[0] >> 16) | (c[1] & 0xffff0000u);
    }
    hi = __builtin_bit_cast(bf16x8_t, h);
    mid = __builtin_bit_cast(bf16x8_t, m);
    lo = __builtin_bit_cast(bf16x8_t, l);
}

// A tile of 16 tokens x 16 experts per workgroup; its four waves take the K
// steps of 32 in turn and their sums meet in LDS.
template <bool WF32>
__global__ void __launch_bounds__(256)
moe_router_logits(mega_moe_router_logits_args a) {
    __shared__ float part[4][16][17];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int r = lane & 15, kq = (lane >> 4) * 8;
    const int e_tiles = (a.num_experts + 15) / 16;
    const int e0 = (int)(blockIdx.x % e_tiles) * 16;
    const int64_t t0 = (int64_t)(blockIdx.x / e_tiles) * 16;
    const int e = e0 + r;
    const int64_t t = t0 + r;
    const int H = a.hidden, E = a.num_experts;
    f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k0 = wave * 32; k0 < H; k0 += 128) {
        const int k = k0 + kq;
        u32x4_t xv = {0u, 0u, 0u, 0u};
        if (t < a.num_tokens && k < H)
            xv = *reinterpret_cast<const u32x4_t*>(a.x + t * a.x_stride + k);
        const bf16x8_t xb = __builtin_bit_cast(bf16x8_t, xv);
        if constexpr (WF32) {
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 0.0f;
            if (e < E && k < H) load8<true>(a.w, (size_t)e * H + k, w);
            bf16x8_t hi, mid, lo;
            split3(w, hi, mid, lo);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, xb, acc, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(mid, xb, acc, 0, 0, 0);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, xb, acc, 0, 0, 0);
        } else {
            u32x4_t wv = {0u, 0u, 0u, 0u};
            if (e < E && k < H)
                wv = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.w) + (size_t)e * H + k);
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, wv), xb, acc, 0, 0, 0);
        }
    }
    // lane l holds experts 4 (l / 16) .. + 3 of token l % 16
#pragma unroll
    for (int i = 0; i < 4; ++i) part[wave][r][(lane >> 4) * 4 + i] = acc[i];
    __syncthreads();
    const int to = threadIdx.x >> 4, eo = threadIdx.x & 15;
    const float s = (part[0][to][eo] + part[1][to][eo]) + (part[2][to][eo] + part[3][to][eo]);
    const int64_t tt = t0 + to;
    const int ee = e0 + eo;
    if (tt < a.num_tokens && ee < E) a.logits[tt * a.logits_stride + ee] = s;
}

// Gradients, each a product over K with tiles of 64 x 64 in float32: DX:
// rows are tokens, columns H, K the experts; else rows are experts, K tokens.
template <bool DX>
__global__ void __launch_bounds__(256)
moe_router_logits_backward(mega_moe_router_logits_args a) {
    __shared__ float sa[16][64 + 4], sb[16][64 + 4];
    const int tid = threadIdx.x;
    const int H = a.hidden, E = a.num_experts;
    const int64_t M = DX ? a.num_tokens : E, K = DX ? E : a.num_tokens;
    const int n_tiles = (H + 63) / 64;
    const int64_t m0 = (int64_t)(blockIdx.x / n_tiles) * 64;
    const int n0 = (int)(blockIdx.x % n_tiles) * 64;
    const int tx = tid & 15, ty = tid >> 4;
    float acc[4][4] = {};
    for (int64_t k0 = 0; k0 < K; k0 += 16) {
        for (int i = tid; i < 1024; i += 256) {
            // dlogits is [T, E]: its rows are contiguous in E
            const int m = DX ? i >> 4 : i & 63, k = DX ? i & 15 : i >> 6;
            const int64_t gm = m0 + m, gk = k0 + k;
            float v = 0.0f;
            if (gm < M && gk < K) v = DX ? a.dlogits[gm * a.dlogits_stride + gk] : a.dlogits[gk * a.dlogits_stride + gm];
            sa[k][m] = v;
            const int n = i & 63, kb = i >> 6;
            const int64_t gkb = k0 + kb;
            float w = 0.0f;
            if (n0 + n < H && gkb < K) {
                if (!DX) w = bf16_value(a.x[gkb * a.x_stride + n0 + n]);
                else if (a.weight_type == MEGA_MOE_F32) w = static_cast<const float*>(a.w)[gkb * H + n0 + n];
                else w = bf16_value(static_cast<const uint16_t*>(a.w)[gkb * H + n0 + n]);
            }
            sb[kb][n] = w;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] += sa[k][ty * 4 + i] * sb[k][tx * 4 + j];
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        if (m >= M) break;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx * 4 + j;
            if (n >= H) break;
            if (DX) {
                float v = acc[i][j];
                if (a.dx_add) v += bf16_value(a.dx_add[m * a.dx_add_stride + n]);
                a.dx[m * a.dx_stride + n] = (uint16_t)bf16_pair(v, 0.0f);
            } else {
                a.dw[m * H + n] = acc[i][j];
            }
        }
    }
}

int64_t router_logits_workspace(const mega_moe_router_logits_args&) { return 0; }

void launch_router_logits(const mega_moe_router_logits_args& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.num_experts + 15) / 16) * (unsigned)((a.num_tokens + 15) / 16));
    if (a.weight_type == MEGA_MOE_F32)
        hipLaunchKernelGGL((moe_router_logits<true>), grid, dim3(256), 0, stream, a);
    else
        hipLaunchKernelGGL((moe_router_logits<false>), grid, dim3(256), 0, stream, a);
}

void launch_router_logits_backward(const mega_moe_router_logits_args& a, hipStream_t stream) {
    const unsigned nx = (unsigned)(a.hidden + 63) / 64;
    if (a.dx && a.num_tokens > 0)
        hipLaunchKernelGGL((moe_router_logits_backward<true>),
                           dim3(nx * ((unsigned)(a.num_tokens + 63) / 64)), dim3(256), 0, stream, a);
    if (a.dw)
        hipLaunchKernelGGL((moe_router_logits_backward<false>),
                           dim3(nx * ((unsigned)(a.num_experts + 63) / 64)), dim3(256), 0, stream, a);
}

}  // namespace mega_moe
