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

// Gradients.  A workgroup is G groups of nt threads, each group on a row of
// its own; group i of workgroup b takes rows b * G + i, then every grid * G-th.
// A thread keeps its eight columns from row to row, and with them its part of
// the sums over tokens, in registers.  At the end the groups' sums meet in LDS
// and the workgroup's go to the workspace, [grid][sums][H] (those that are
// asked for), where moe_norm_reduce adds them up in order.
//
// Memory bound: the next row's loads stay in flight over the two row sums (the
// barriers would leave the memory idle otherwise), and the weights lie in LDS.
template <bool SF32, bool FULL>
__global__ void __launch_bounds__(1024)
moe_norm_backward(mega_moe_norm_backward_args a, float* ws, int nt) {
    extern __shared__ float shared[];            // the weights, [3][H]; then a group's sums
    __shared__ float part1[16][3];
    __shared__ float part2[16][2];
    const int group = threadIdx.x / nt, tid = threadIdx.x - group * nt, G = blockDim.x / nt;
    const int H = a.hidden, col = tid * 8;
    const bool in = col < H;
    const float inv_h = 1.0f / (float)H;
    const bool normed = a.y && a.post_weight;
    constexpr int SW = SF32 ? 2 : 1;
    const u32x4_t none = {0u, 0u, 0u, 0u};
    u32x4_t raw_r[SW], raw_dr[SW], raw_dn, raw_y;
    float raw_tg = 1.0f;

    const auto fetch = [&](int64_t t) {
        const bool live = in && t < a.num_tokens;
#pragma unroll
        for (int i = 0; i < SW; ++i) {
            raw_r[i] = raw_dr[i] = none;
            if (live && a.dn) raw_r[i] = raw8<SF32>(a.r, t * a.r_stride + col)[i];
            if (live && a.dr && !SF32) raw_dr[i] = raw8<SF32>(a.dr, t * a.dr_stride + col)[i];
        }
        raw_dn = raw_y = none;
        if (live && a.dn) raw_dn = raw8<false>(a.dn, t * a.dn_stride + col)[0];
        if (live && a.y) raw_y = raw8<false>(a.y, t * a.y_stride + col)[0];
        if (!FULL && a.gate_kind == MEGA_MOE_GATE_TOKEN && t < a.num_tokens) {
            raw_tg = a.gate_type == MEGA_MOE_F32 ? static_cast<const float*>(a.gate)[t]
                                                 : bf16_value(static_cast<const uint16_t*>(a.gate)[t]);
        }
    };
    // the pre weight, the post weight and a gate by channel: 1 where there is none
    const void* channel = a.gate_kind == MEGA_MOE_GATE_CHANNEL ? a.gate : nullptr;
    for (int c = threadIdx.x * 8; c < H; c += blockDim.x * 8)
        for (int which = 0; which < 3; ++which) {
            const void* p = which == 0 ? a.pre_weight : which == 1 ? a.post_weight : channel;
            float w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = 1.0f;
            if (p) load8(p, which == 2 ? a.gate_type : a.weight_type, c, w);
            store8<true>(shared, (size_t)which * H + c, w);
        }
    const auto weight = [&](int which, float (&w)[8]) {
        if (in) load8<true>(shared, (size_t)which * H + col, w);
    };

    float s_pre[8], s_post[8], s_gate[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) s_pre[i] = s_post[i] = s_gate[i] = 0.0f;

    // every group makes the same number of rounds: the barriers are shared
    const int64_t step = (int64_t)gridDim.x * G;
    int64_t t = (int64_t)blockIdx.x * G + group;
    const int64_t rounds = (a.num_tokens - (int64_t)blockIdx.x * G + step - 1) / step;
    fetch(t);
    __syncthreads();
    for (int64_t round = 0; round < rounds; ++round, t += step) {
        const bool live = in && t < a.num_tokens;
        // this row stays packed until its values are needed
        float g[8];
        u32x4_t cur_r[SW], cur_g[2];
        values8<SF32>(raw_dr, g);
#pragma unroll
        for (int i = 0; i < SW; ++i) cur_r[i] = raw_r[i];
        const u32x4_t cur_dn = raw_dn, cur_y = raw_y;
        // what is needed after the first sum only, and would not fit beside the
        // next row's registers, is loaded now
        cur_g[0] = cur_g[1] = none;
        if (FULL && live) {
            if (a.gate_type == MEGA_MOE_F32) {
                cur_g[0] = raw8<true>(a.gate, t * a.gate_stride + col)[0];
                cur_g[1] = raw8<true>(a.gate, t * a.gate_stride + col)[1];
            } else {
                cur_g[0] = raw8<false>(a.gate, t * a.gate_stride + col)[0];
            }
        }
        if (SF32 && live && a.dr) load8<true>(a.dr, t * a.dr_stride + col, g);
        const float tg = raw_tg;
        if (round + 1 < rounds) fetch(t + step);
        // the sums that both norms need: of r^2 and u r, and of y^2
        float s1[3] = {0.0f, 0.0f, 0.0f};
        {
            float w[8] = {}, r[8], u[8], y[8];
            weight(0, w);
            values8<SF32>(cur_r, r);
            unpack8(cur_dn, u);
            unpack8(cur_y, y);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s1[0] += r[i] * r[i];
                s1[1] += u[i] * w[i] * r[i];
                s1[2] += y[i] * y[i];
            }
        }
        group_sum(s1, part1, group, nt);
        if (a.dn) {
            const float rs = rsqrtf(s1[0] * inv_h + a.pre_eps);
            const float mean = s1[1] * rs * inv_h;       // mean of u * rh
            float w[8] = {}, r[8], u[8];
            weight(0, w);
            values8<SF32>(cur_r, r);
            unpack8(cur_dn, u);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float rh = r[i] * rs;
                g[i] += rs * (u[i] * w[i] - rh * mean);
                // a group that is out of rows has u = 0, but rh may be infinite
                if (live) s_pre[i] += u[i] * rh;
            }
        }
        if (a.dh && live) {
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = a.residual_scale * g[i];
            store8<SF32>(a.dh, t * a.dh_stride + col, o);
        }
        if (a.y) {
            const float ys = normed ? rsqrtf(s1[2] * inv_h + a.post_eps) : 1.0f;
            float s2[2] = {0.0f, 0.0f};
            {
                // g becomes v = gate * g * post_weight
                float w[8] = {}, ga[8] = {}, dg[8], y[8];
                weight(1, w);
                if constexpr (FULL) {
                    if (a.gate_type == MEGA_MOE_F32) values8<true>(cur_g, ga);
                    else unpack8(cur_g[0], ga);
                } else {
                    weight(2, ga);
                }
                unpack8(cur_y, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] *= ys;
                    dg[i] = y[i] * w[i] * g[i];
                    const float dz = (FULL ? ga[i] : ga[i] * tg) * g[i];
                    if (live) {
                        s_post[i] += dz * y[i];
                        if (!FULL) s_gate[i] += dg[i];
                    }
                    g[i] = dz * w[i];
                    s2[0] += g[i] * y[i];
                    s2[1] += dg[i];
                }
                if (FULL && a.dgate && live) store8(a.dgate, a.gate_type, t * a.dgate_stride + col, dg);
            }
            const bool token_grad = !FULL && a.gate_kind == MEGA_MOE_GATE_TOKEN && a.dgate;
            if (normed || token_grad) group_sum(s2, part2, group, nt);
            if (token_grad && tid == 0 && t < a.num_tokens) static_cast<float*>(a.dgate)[t] = s2[1];
            if (a.dy && live) {
                const float mean = normed ? s2[0] * inv_h : 0.0f;
                float o[8], y[8];
                unpack8(cur_y, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = ys * (g[i] - y[i] * ys * mean);
                store8<false>(a.dy, t * a.dy_stride + col, o);
            }
        }
        // part1 is written again by the next round: every wave has left it
        __syncthreads();
    }
    // nothing reads the weights any more (the last round ended in a barrier)
    int k = 0;
    const auto put = [&](float (&s)[8]) {
        // the groups in turn, onto the first one's sums
        for (int q = 1; q < G; ++q) {
            if (group == q && in) store8<true>(shared, (size_t)col, s);
            __syncthreads();
            if (group == 0 && in) {
                float o[8];
                load8<true>(shared, (size_t)col, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] += o[i];
            }
            __syncthreads();
        }
        if (group == 0 && in) store8<true>(ws, ((size_t)blockIdx.x * norm_sums(a) + k) * H + col, s);
        ++k;
    };
    if (a.dpre_weight) put(s_pre);
    if (a.dpost_weight) put(s_post);
    if (!FULL && a.gate_kind == MEGA_MOE_GATE_CHANNEL && a.dgate) put(s_gate);
}

// Adds the workgroups' sums: 64 columns of one sum per workgroup; its eight
// waves take every eighth row each, and meet in LDS.
__global__ void __launch_bounds__(512)
moe_norm_reduce(const float* ws, float* out0, float* out1, float* out2, int H, int rows) {
    __shared__ float part[8][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int col = blockIdx.x * 64 + lane, sums = gridDim.y;
    float* out = blockIdx.y == 0 ? out0 : blockIdx.y == 1 ? out1 : out2;
    const float* p = ws + (size_t)blockIdx.y * H + col;
    const size_t pitch = (size_t)sums * H;
    float s = 0.0f;
    if (col < H) {
#pragma unroll 8
        for (int i = wave; i < rows; i += 8) s += p[i * pitch];
    }
    part[wave][lane] = s;
    __syncthreads();
    if (wave || col >= H) return;
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) s += part[w][lane];
    out[col] = s;
}

namespace {
int chunks(int H) { return H <= 2048 ? 1 : 2; }
unsigned threads(int H, int c) { return (unsigned)((H / 8 + c - 1) / c + 63) / 64 * 64; }
}  // namespace

void launch_norm(const mega_moe_norm_args& a, hipStream_t stream) {
    const int c = chunks(a.hidden);
    const dim3 grid((unsigned)a.num_tokens), block(threads(a.hidden, c));
    const bool f = a.stream_type == MEGA_MOE_F32;
#define NORM(CC)                                                                             \
    if (f) hipLaunchKernelGGL((moe_norm<true, CC>), grid, block, 0, stream, a);              \
    else hipLaunchKernelGGL((moe_norm<false, CC>), grid, block, 0, stream, a)
    if (c == 1) { NORM(1); } else { NORM(2); }
#undef NORM
}

// The backward kernel: a chunk per thread, and as many row groups as fit into
// 1024 threads.
namespace {
int row_groups(int H) { return 1024 / (int)threads(H, 1); }
}  // namespace

int norm_backward_blocks(int tokens, int hidden) {
    const int g = row_groups(hidden);
    const int need = (tokens + g - 1) / g;
    return need < 256 ? need : 256;
}

void launch_norm_backward(const mega_moe_norm_backward_args& a, hipStream_t stream) {
    const int nt = (int)threads(a.hidden, 1), groups = row_groups(a.hidden);
    const int rows = norm_backward_blocks(a.num_tokens, a.hidden);
    const int n = norm_sums(a);
    float* ws = static_cast<float*>(a.workspace);
    if (rows > 0) {
        const auto go = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, dim3((unsigned)rows), dim3((unsigned)(nt * groups)), (unsigned)a.hidden * 12,
                               stream, a, ws, nt);
        };
        const bool f = a.stream_type == MEGA_MOE_F32, full = a.gate_kind == MEGA_MOE_GATE_FULL;
        if (full && f) go(moe_norm_backward<true, true>);
        else if (full) go(moe_norm_backward<false, true>);
        else if (f) go(moe_norm_backward<true, false>);
        else go(moe_norm_backward<false, false>);
    }
    if (n) {
        float* outs[3];
        int k = 0;
        if (a.dpre_weight) outs[k++] = a.dpre_weight;
        if (a.dpost_weight) outs[k++] = a.dpost_weight;
        if (a.gate_kind == MEGA_MOE_GATE_CHANNEL && a.dgate) outs[k++] = static_cast<float*>(a.dgate);
        hipLaunchKernelGGL(moe_norm_reduce, dim3((unsigned)(a.hidden + 63) / 64, (unsigned)n), dim3(512), 0, stream, ws,
                           outs[0], n > 1 ? outs[1] : nullptr, n > 2 ? outs[2] : nullptr, a.hidden, rows);
    }
}

}  // namespace mega_moe
