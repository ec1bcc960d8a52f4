// The norms before and after a block, fused with its gate, the residual stream
// and the layer's E4M3 input, and their gradients.
#include <hip/hip_runtime.h>

#include "block_util.h"
#include "norm.h"

namespace mega_moe {

// One workgroup per token; thread i holds columns 8 (c * threads + i) .. + 7
// for its C chunks, so the whole row stays in registers between its loads and
// its stores.  Memory bound: every tensor is read or written once.
template <bool SF32, int C>
__global__ void __launch_bounds__(1024)
moe_norm(mega_moe_norm_args a) {
    __shared__ float part[2][16][1];
    const int nt = blockDim.x, tid = threadIdx.x;
    const size_t t = blockIdx.x;
    const int H = a.hidden;
    const float inv_h = 1.0f / (float)H;
    float r[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c * nt + tid) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) r[c][i] = 0.0f;
        if (col < H) load8<SF32>(a.h, t * a.h_stride + col, r[c]);
    }
    if (a.y) {
        float z[C][8];
        float s[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * nt + tid) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) z[c][i] = 0.0f;
            if (col < H) load8<false>(a.y, t * a.y_stride + col, z[c]);
        }
        float ys = 1.0f;
        if (a.post_weight) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) s[0] += z[c][i] * z[c][i];
            block_sum(s, part[0]);
            ys = rsqrtf(s[0] * inv_h + a.post_eps);
        }
        float tg = 1.0f;
        if (a.gate_kind == MEGA_MOE_GATE_TOKEN)
            tg = a.gate_type == MEGA_MOE_F32 ? static_cast<const float*>(a.gate)[t]
                                             : bf16_value(static_cast<const uint16_t*>(a.gate)[t]);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * nt + tid) * 8;
            if (col >= H) continue;
            if (a.post_weight) {
                float w[8];
                load8(a.post_weight, a.weight_type, col, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[c][i] = z[c][i] * ys * w[i];
            }
            if (a.gate_kind >= MEGA_MOE_GATE_CHANNEL) {
                float g[8];
                load8(a.gate, a.gate_type,
                      a.gate_kind == MEGA_MOE_GATE_FULL ? t * a.gate_stride + col : (size_t)col, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[c][i] *= g[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) r[c][i] = a.residual_scale * r[c][i] + tg * z[c][i];
        }
    }
    if (a.r) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * nt + tid) * 8;
            if (col < H) store8<SF32>(a.r, t * a.r_stride + col, r[c]);
        }
    }
    if (!a.pre_weight) return;
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += r[c][i] * r[c][i];
    block_sum(s, part[1]);
    const float rs = rsqrtf(s[0] * inv_h + a.pre_eps);
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = (c * nt + tid) * 8;
        float n[8];
        uint32_t m = 0;
        if (col < H) {
            float w[8];
            load8(a.pre_weight, a.weight_type, col, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                n[i] = r[c][i] * rs * w[i];
                // magnitudes compared as integers: a NaN is the largest
                m = max(m, __float_as_uint(n[i]) & 0x7fffffffu);
            }
            if (a.n) store8<false>(a.n, t * a.n_stride + col, n);
        }
        if (a.q) {
            // 16 lanes hold one block of 128 columns (H is a multiple of 128)
#pragma unroll
            for (int d = 1; d < 16; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
            if (col < H) {
                const float amax = __uint_as_float(m);
                const float sf = amax / 448.0f;
                // tiny blocks are scaled up first, so that the reciprocal is finite
                const float up = sf < 0x1p-100f ? 0x1p100f : 1.0f;
                const float inv = amax == 0.0f ? 0.0f : 1.0f / ((amax * up) / 448.0f);
                float v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = n[i] * up * inv;
                int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
                lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
                int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
                hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
                *reinterpret_cast<int2*>(a.q + t * H + col) = int2{lo, hi};
                if ((tid & 15) == 0) a.q_sf[t * (H / 128) + col / 128] = sf;
            }
        }
    }
}

// Gradients.  A workgroup takes rows b, b + grid, ..., one at a time; its
// threads keep their columns, and with them their part of the sums over
// tokens, in registers; each workgroup's sums go to the workspace, [grid][3][H]
// (those that are asked for), and moe_norm_reduce adds them up in order.
template <bool SF32, int C>
__global__ void __launch_bounds__(1024)
moe_norm_backward(mega_moe_norm_backward_args a, float* ws) {
    __shared__ float part1[16][3];
    __shared__ float part2[16][2];
    const int nt = blockDim.x, tid = threadIdx.x;
    const int H = a.hidden;
    const float inv_h = 1.0f / (float)H;
    const bool normed = a.y && a.post_weight;
    float s_pre[C][8], s_post[C][8], s_gate[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) s_pre[c][i] = s_post[c][i] = s_gate[c][i] = 0.0f;
    for (int64_t t = blockIdx.x; t < a.num_tokens; t += gridDim.x) {
        float g[C][8], r[C][8], u[C][8], y[C][8];
        float s1[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * nt + tid) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) g[c][i] = r[c][i] = u[c][i] = y[c][i] = 0.0f;
            if (col >= H) continue;
            if (a.dr) load8<SF32>(a.dr, t * a.dr_stride + col, g[c]);
            if (a.dn) {
                load8<SF32>(a.r, t * a.r_stride + col, r[c]);
                load8<false>(a.dn, t * a.dn_stride + col, u[c]);
            }
            if (a.y) load8<false>(a.y, t * a.y_stride + col, y[c]);
        }
        // the sums that both norms need: of r^2 and u r, and of y^2
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * nt + tid) * 8;
            if (col >= H) continue;
            if (a.dn) {
                float w[8];
                load8(a.pre_weight, a.weight_type, col, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    s1[0] += r[c][i] * r[c][i];
                    s1[1] += u[c][i] * w[i] * r[c][i];
                }
            }
            if (normed) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s1[2] += y[c][i] * y[c][i];
            }
        }
        block_sum(s1, part1);
        if (a.dn) {
            const float rs = rsqrtf(s1[0] * inv_h + a.pre_eps);
            const float mean = s1[1] * rs * inv_h;       // mean of u * rh
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int col = (c * nt + tid) * 8;
                if (col >= H) continue;
                float w[8];
                load8(a.pre_weight, a.weight_type, col, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float rh = r[c][i] * rs;
                    g[c][i] += rs * (u[c][i] * w[i] - rh * mean);
                    s_pre[c][i] += u[c][i] * rh;
                }
            }
        }
        if (a.dh) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int col = (c * nt + tid) * 8;
                float o[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = a.residual_scale * g[c][i];
                if (col < H) store8<SF32>(a.dh, t * a.dh_stride + col, o);
            }
        }
        if (a.y) {
            const float ys = normed ? rsqrtf(s1[2] * inv_h + a.post_eps) : 1.0f;
            float tg = 1.0f;
            if (a.gate_kind == MEGA_MOE_GATE_TOKEN)
                tg = a.gate_type == MEGA_MOE_F32 ? static_cast<const float*>(a.gate)[t]
                                                 : bf16_value(static_cast<const uint16_t*>(a.gate)[t]);
            float s2[2] = {0.0f, 0.0f};
            // g becomes v = gate * g * post_weight, y becomes yh
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int col = (c * nt + tid) * 8;
                if (col >= H) continue;
                float w[8], ga[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = 1.0f, ga[i] = tg;
                if (normed) load8(a.post_weight, a.weight_type, col, w);
                if (a.gate_kind >= MEGA_MOE_GATE_CHANNEL)
                    load8(a.gate, a.gate_type,
                          a.gate_kind == MEGA_MOE_GATE_FULL ? t * a.gate_stride + col : (size_t)col,
                          ga);
                float dg[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[c][i] *= ys;
                    dg[i] = y[c][i] * w[i] * g[c][i];
                    const float dz = ga[i] * g[c][i];
                    s_post[c][i] += dz * y[c][i];
                    g[c][i] = dz * w[i];
                    s2[0] += g[c][i] * y[c][i];
                    s2[1] += dg[i];
                    s_gate[c][i] += dg[i];
                }
                if (a.gate_kind == MEGA_MOE_GATE_FULL && a.dgate)
                    store8(a.dgate, a.gate_type, t * a.dgate_stride + col, dg);
            }
            const bool token_grad = a.gate_kind == MEGA_MOE_GATE_TOKEN && a.dgate;
            if (normed || token_grad) block_sum(s2, part2);
            if (token_grad && tid == 0) static_cast<float*>(a.dgate)[t] = s2[1];
            if (a.dy) {
                const float mean = normed ? s2[0] * inv_h : 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const int col = (c * nt + tid) * 8;
                    float o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = ys * (g[c][i] - y[c][i] * mean);
                    if (col < H) store8<false>(a.dy, t * a.dy_stride + col, o);
                }
            }
        }
        // part1 is written again by the next row: every wave has left it
        __syncthreads();
    }
    int k = 0;
    const auto put = [&](const float (&s)[C][8]) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int col = (c * nt + tid) * 8;
            if (col < H) store8<true>(ws, ((size_t)blockIdx.x * norm_sums(a) + k) * H + col, s[c]);
        }
        ++k;
    };
    if (a.dpre_weight) put(s_pre);
    if (a.dpost_weight) put(s_post);
    if (a.gate_kind == MEGA_MOE_GATE_CHANNEL && a.dgate) put(s_gate);
}

// Adds the workgroups' sums: 64 columns per workgroup, four threads each, a
// quarter of the rows apiece.
__global__ void __launch_bounds__(256)
moe_norm_reduce(mega_moe_norm_backward_args a, const float* ws, int rows) {
    __shared__ float part[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = norm_sums(a);
    const int col = blockIdx.x * 64 + lane;      // of the n * H sums
    float s = 0.0f;
    if (col < n * a.hidden)
        for (int i = wave; i < rows; i += 4) s += ws[(size_t)i * n * a.hidden + col];
    part[wave][lane] = s;
    __syncthreads();
    if (wave || col >= n * a.hidden) return;
    s = (part[0][lane] + part[1][lane]) + (part[2][lane] + part[3][lane]);
    float* outs[3];
    int k = 0;
    if (a.dpre_weight) outs[k++] = a.dpre_weight;
    if (a.dpost_weight) outs[k++] = a.dpost_weight;
    if (a.gate_kind == MEGA_MOE_GATE_CHANNEL && a.dgate) outs[k++] = static_cast<float*>(a.dgate);
    const int which = col / a.hidden;
    float* out = which == 0 ? outs[0] : which == 1 ? outs[1] : outs[2];
    out[col - which * a.hidden] = s;
}

namespace {
int chunks(int H) { return H <= 2048 ? 1 : H <= 8192 ? 2 : 4; }
unsigned threads(int H, int c) { return (unsigned)((H / 8 + c - 1) / c + 63) / 64 * 64; }
}  // namespace

void launch_norm(const mega_moe_norm_args& a, hipStream_t stream) {
    const int c = chunks(a.hidden);
    const dim3 grid((unsigned)a.num_tokens), block(threads(a.hidden, c));
    const bool f = a.stream_type == MEGA_MOE_F32;
#define NORM(CC)                                                                             \
    if (f) hipLaunchKernelGGL((moe_norm<true, CC>), grid, block, 0, stream, a);              \
    else hipLaunchKernelGGL((moe_norm<false, CC>), grid, block, 0, stream, a)
    if (c == 1) { NORM(1); } else if (c == 2) { NORM(2); } else { NORM(4); }
#undef NORM
}

int norm_backward_blocks(int tokens) { return tokens < 512 ? tokens : 512; }

void launch_norm_backward(const mega_moe_norm_backward_args& a, hipStream_t stream) {
    const int c = chunks(a.hidden);
    const int rows = norm_backward_blocks(a.num_tokens);
    const dim3 grid((unsigned)rows), block(threads(a.hidden, c));
    const bool f = a.stream_type == MEGA_MOE_F32;
    float* ws = static_cast<float*>(a.workspace);
#define NORM(CC)                                                                                 \
    if (f) hipLaunchKernelGGL((moe_norm_backward<true, CC>), grid, block, 0, stream, a, ws);     \
    else hipLaunchKernelGGL((moe_norm_backward<false, CC>), grid, block, 0, stream, a, ws)
    if (rows > 0) {
        if (c == 1) { NORM(1); } else if (c == 2) { NORM(2); } else { NORM(4); }
    }
#undef NORM
    const int n = norm_sums(a);
    if (n)
        hipLaunchKernelGGL(moe_norm_reduce, dim3((unsigned)(n * a.hidden + 63) / 64), dim3(256), 0,
                           stream, a, ws, rows);
}

}  // namespace mega_moe
