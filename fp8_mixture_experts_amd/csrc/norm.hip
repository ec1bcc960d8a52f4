// The norms before and after a block, fused with its gate, the residual stream
// and the layer's E4M3 input, and their gradients.
#include <hip/hip_runtime.h>

#include "block_util.h"
#include "norm.h"

namespace mega_moe {

// A workgroup is G groups of nt threads, each group on a row of its own; group
// i of workgroup b takes rows b * G + i, then every grid * G-th.  A thread keeps
// its eight columns, and their weights, from row to row, and a row stays in
// registers between its loads and its stores.
//
// Memory bound: every tensor is read or written once.  The next row's loads
// stay in flight over the two row sums; two rows at a time for a group took as
// long with half as many registers again.  The weights are read once per
// workgroup: read again for each row they were 40% more bytes to the compute
// units than the rows.  r is read again after the whole layer and streamed past
// the caches, n and q are read next and are not: with the readers behind it, and
// 256 MiB between r and its reader, 249 us, against 253 with nothing streamed and
// 259 with n streamed too.  8192 rows of 7168 in BF16 with y, a gate by channel
// and all three outputs: 96 to 98 us, 5.5 TB/s (a copy of 1 GiB: 5.1 TB/s; part of
// the 530 MB stays in the last-level cache); the codes' exact quotients are 1 us of
// it. 577 rows of 4096 in float32: 7.5 to 7.9 us.
template <bool SF32, bool FULL>
__global__ void __launch_bounds__(1024)
moe_norm(mega_moe_norm_args a, int nt) {
    __shared__ float part[2][2][16][1];          // by round: one is read while the next is written
    // a group is whole waves: its number, and with it the row, is the same for a wave
    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / nt);
    const int tid = threadIdx.x - group * nt, G = blockDim.x / nt;
    const int H = a.hidden, col = tid * 8;
    const bool in = col < H;
    const float inv_h = 1.0f / (float)H;
    const u32x4_t none = {0u, 0u, 0u, 0u};
    u32x4_t raw_h0 = none, raw_h1 = none, raw_y = none, raw_g0 = none, raw_g1 = none;
    float raw_tg = 1.0f;

    const auto fetch = [&](int64_t t) {
        const bool live = in && t < a.num_tokens;
        if (live) {
            raw_h0 = raw8<SF32>(a.h, t * a.h_stride + col)[0];
            if (SF32) raw_h1 = raw8<SF32>(a.h, t * a.h_stride + col)[1];
        }
        if (live && a.y) raw_y = raw8<false>(a.y, t * a.y_stride + col)[0];
        if constexpr (FULL) {
            if (live && a.gate_type == MEGA_MOE_F32) {
                raw_g0 = raw8<true>(a.gate, t * a.gate_stride + col)[0];
                raw_g1 = raw8<true>(a.gate, t * a.gate_stride + col)[1];
            } else if (live) {
                raw_g0 = raw8<false>(a.gate, t * a.gate_stride + col)[0];
            }
        } else if (a.gate_kind == MEGA_MOE_GATE_TOKEN && t < a.num_tokens) {
            raw_tg = a.gate_type == MEGA_MOE_F32 ? static_cast<const float*>(a.gate)[t]
                                                 : bf16_value(static_cast<const uint16_t*>(a.gate)[t]);
        }
    };
    const int64_t step = (int64_t)gridDim.x * G;
    int64_t t = (int64_t)blockIdx.x * G + group;
    const int64_t rounds = (a.num_tokens - (int64_t)blockIdx.x * G + step - 1) / step;
    fetch(t);
    // the pre weight, and the post weight times a gate by channel
    float w_pre[8], w_post[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w_pre[i] = w_post[i] = 1.0f;
    if (in && a.pre_weight) load8(a.pre_weight, a.weight_type, col, w_pre);
    if (in && a.post_weight) load8(a.post_weight, a.weight_type, col, w_post);
    if (in && a.gate_kind == MEGA_MOE_GATE_CHANNEL) {
        float g[8];
        load8(a.gate, a.gate_type, col, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) w_post[i] *= g[i];
    }
    for (int64_t round = 0; round < rounds; ++round, t += step) {
        const bool live = in && t < a.num_tokens;
        float r[8];
        values8<SF32>(raw_h0, raw_h1, r);
        const u32x4_t cur_y = raw_y, cur_g0 = raw_g0, cur_g1 = raw_g1;
        const float tg = raw_tg;
        if (round + 1 < rounds) fetch(t + step);
        if (a.y) {
            float z[8], s[1] = {0.0f};
            unpack8(cur_y, z);
            float ys = tg;
            if (a.post_weight) {
#pragma unroll
                for (int i = 0; i < 8; ++i) s[0] += z[i] * z[i];
                group_sum(s, part[round & 1][0], group, nt);
                ys = rsqrtf(s[0] * inv_h + a.post_eps) * tg;
            }
            if constexpr (FULL) {
                float g[8];
                if (a.gate_type == MEGA_MOE_F32) values8<true>(cur_g0, cur_g1, g);
                else unpack8(cur_g0, g);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] *= g[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = a.residual_scale * r[i] + z[i] * ys * w_post[i];
        }
        if (a.r && live) stream8<SF32>(a.r, t * a.r_stride + col, r);
        if (!a.pre_weight) continue;
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) s[0] += r[i] * r[i];
        group_sum(s, part[round & 1][1], group, nt);
        const float rs = rsqrtf(s[0] * inv_h + a.pre_eps);
        float n[8];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            n[i] = r[i] * rs * w_pre[i];
            // magnitudes compared as integers: a NaN is the largest
            m = max(m, __float_as_uint(n[i]) & 0x7fffffffu);
        }
        if (a.n && live) store8<false>(a.n, t * a.n_stride + col, n);
        if (!a.q) continue;
        // 16 lanes hold one block of 128 columns (H is a multiple of 128)
        m = over_lanes<16>(m, [](uint32_t x, uint32_t y) { return x > y ? x : y; });
        if (!live) continue;
        const float amax = __uint_as_float(m);
        const float sf = amax / 448.0f;
        // tiny blocks are scaled up first, so that the reciprocal is finite
        const float up = sf < 0x1p-100f ? 0x1p100f : 1.0f;
        float d = (amax * up) / 448.0f;
        const float inv = amax == 0.0f ? 0.0f : 1.0f / d;
        if (inv == 0.0f) d = 0.0f;               // a scale of 0 or infinity: codes of 0
        // The quotient n / d: the product with the reciprocal is off by up to a step and
        // a half, and next to a tie takes another code; one step of Newton's iteration
        // (the exact remainder, times the reciprocal) rounds it as a division does.
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = n[i] * up, q = x * inv;
            v[i] = fmaf(-fmaf(q, d, -x), inv, q);
        }
        int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], lo, true);
        int hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4], v[5], 0, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6], v[7], hi, true);
        *reinterpret_cast<int2*>(a.q + t * H + col) = int2{lo, hi};
        if ((tid & 15) == 0) a.q_sf[t * (H / 128) + col / 128] = sf;
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
// dh waits for the whole layer's gradients before it is read and is streamed past
// the caches, dy is read next and is not: with a reader of dy behind it 58 us
// against 60 (BF16, a gate by channel), a full gate as long, float32 with one 91
// against 89.  4096 rows of 4096, all gradients: BF16 and a gate by channel 41 to 42
// us, 4.8 TB/s (201 MB), a full gate in BF16 50 to 53, 5.1 TB/s (268 MB); float32 58
// to 59, 5.1 TB/s (302 MB), with a full gate in BF16 70 to 72, 5.1 TB/s (369 MB), and
// 36 bytes of scratch a lane.  The sums over the rows take 4 to 5 us more.
template <bool SF32, bool FULL>
__global__ void __launch_bounds__(1024)
moe_norm_backward(mega_moe_norm_backward_args a, float* ws, int nt) {
    extern __shared__ float shared[];            // the weights, [3][H]; then a group's sums
    __shared__ float part1[16][3];
    __shared__ float part2[16][2];
    // a group is whole waves: its number, and with it the row, is the same for a wave
    const int group = __builtin_amdgcn_readfirstlane(threadIdx.x / nt);
    const int tid = threadIdx.x - group * nt, G = blockDim.x / nt;
    const int H = a.hidden, col = tid * 8;
    const bool in = col < H;
    const float inv_h = 1.0f / (float)H;
    const bool normed = a.y && a.post_weight;
    const u32x4_t none = {0u, 0u, 0u, 0u};
    struct Row {
        u32x4_t r0, r1, dr, dn, y;
        float tg;
    } next;

    const auto fetch = [&](Row& w, int64_t t) {
        w.r0 = w.r1 = w.dr = w.dn = w.y = none;
        w.tg = 1.0f;
        if (t >= a.num_tokens) return;
        if (!FULL && a.gate_kind == MEGA_MOE_GATE_TOKEN)
            w.tg = a.gate_type == MEGA_MOE_F32 ? static_cast<const float*>(a.gate)[t]
                                               : bf16_value(static_cast<const uint16_t*>(a.gate)[t]);
        if (!in) return;
        if (a.dn) {
            w.r0 = raw8<SF32>(a.r, t * a.r_stride + col)[0];
            if (SF32) w.r1 = raw8<SF32>(a.r, t * a.r_stride + col)[1];
            w.dn = raw8<false>(a.dn, t * a.dn_stride + col)[0];
        }
        if (a.dr && !SF32) w.dr = raw8<false>(a.dr, t * a.dr_stride + col)[0];
        if (a.y) w.y = raw8<false>(a.y, t * a.y_stride + col)[0];
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
    fetch(next, t);
    __syncthreads();
    for (int64_t round = 0; round < rounds; ++round, t += step) {
        const bool live = in && t < a.num_tokens;
        // this row stays packed until its values are needed
        float g[8];
        unpack8(next.dr, g);
        const u32x4_t cur_r0 = next.r0, cur_r1 = next.r1, cur_dn = next.dn, cur_y = next.y;
        // what is needed after the first sum only, and would not fit beside the
        // next row's registers, is loaded now
        u32x4_t cur_g0 = none, cur_g1 = none;
        if (FULL && live) {
            if (a.gate_type == MEGA_MOE_F32) {
                cur_g0 = raw8<true>(a.gate, t * a.gate_stride + col)[0];
                cur_g1 = raw8<true>(a.gate, t * a.gate_stride + col)[1];
            } else {
                cur_g0 = raw8<false>(a.gate, t * a.gate_stride + col)[0];
            }
        }
        if (SF32 && live && a.dr) load8<true>(a.dr, t * a.dr_stride + col, g);
        const float tg = next.tg;
        if (round + 1 < rounds) fetch(next, t + step);
        // the sums that both norms need: of r^2 and u r, and of y^2
        float s1[3] = {0.0f, 0.0f, 0.0f};
        {
            float w[8] = {}, r[8], u[8], y[8];
            weight(0, w);
            values8<SF32>(cur_r0, cur_r1, r);
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
            values8<SF32>(cur_r0, cur_r1, r);
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
            stream8<SF32>(a.dh, t * a.dh_stride + col, o);
        }
        if (a.y) {
            const float ys = normed ? rsqrtf(s1[2] * inv_h + a.post_eps) : 1.0f;
            float s2[2] = {0.0f, 0.0f};
            {
                // g becomes v = gate * g * post_weight
                float w[8] = {}, ga[8] = {}, dg[8], y[8];
                weight(1, w);
                if constexpr (FULL) {
                    if (a.gate_type == MEGA_MOE_F32) values8<true>(cur_g0, cur_g1, ga);
                    else unpack8(cur_g0, ga);
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
                if (FULL && a.dgate && live) stream8(a.dgate, a.gate_type, t * a.dgate_stride + col, dg);
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
// Threads of a row: eight columns each, whole waves.
int row_threads(int H) { return (H / 8 + 63) / 64 * 64; }
// Rows at a time in a workgroup of up to 1024 threads.
int row_groups(int H) { return 1024 / row_threads(H); }

// Workgroups of the norm for many rows: one to a compute unit, each with a row or
// more in flight.  Two to a unit measured 101 us against 96 (8192 rows of 7168, gate by
// channel, E4M3 output) and 85 against 82 (no gate, no codes).
constexpr int NORM_BLOCKS = 256;
}  // namespace

void launch_norm(const mega_moe_norm_args& a, hipStream_t stream) {
    const int nt = row_threads(a.hidden);
    // no more rows to a workgroup than leave every compute unit some
    const int most = (a.num_tokens + NORM_BLOCKS - 1) / NORM_BLOCKS;
    int groups = most < row_groups(a.hidden) ? most : row_groups(a.hidden);
    int limit = NORM_BLOCKS;
    // Where all rows are on their way at once, three or more to a compute unit (24
    // waves), each has a workgroup of its own: 700 x 4096 8.2 us against 9.3, 3000 x
    // 1024 8.2 against 9.4; at two to a unit it is slower, 400 x 5120 7.2 against 6.8.
    const int together = 24 / (nt / 64);
    if (together >= 3 && a.num_tokens <= NORM_BLOCKS * together) {
        groups = 1;
        limit = a.num_tokens;
    }
    const int blocks = (a.num_tokens + groups - 1) / groups;
    const auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3((unsigned)(blocks < limit ? blocks : limit)),
                           dim3((unsigned)(nt * groups)), 0, stream, a, nt);
    };
    const bool f = a.stream_type == MEGA_MOE_F32, full = a.gate_kind == MEGA_MOE_GATE_FULL;
    if (full && f) go(moe_norm<true, true>);
    else if (full) go(moe_norm<false, true>);
    else if (f) go(moe_norm<true, false>);
    else go(moe_norm<false, false>);
}

int norm_backward_blocks(int tokens, int hidden) {
    const int g = row_groups(hidden);
    const int need = (tokens + g - 1) / g;
    return need < 256 ? need : 256;
}

void launch_norm_backward(const mega_moe_norm_backward_args& a, hipStream_t stream) {
    const int nt = row_threads(a.hidden), groups = row_groups(a.hidden);
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
