// Host side of the dense path next to the layer (the last part of
// include/mega_moe.h): argument checks and launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "checks.h"
#include "mega_moe.h"
#include "product.h"
#include "quantize.h"
#include "rotary.h"

using namespace mega_moe;

namespace {

constexpr int32_t MAX_COLUMNS = 1 << 17;
constexpr int64_t MAX_SF_STRIDE = 1 << 20;      // a tile's scales within 32-bit byte offsets
constexpr int32_t MAX_HEADS = 1024;
constexpr int64_t MAX_HEAD_STRIDE = 1 << 20;
constexpr int32_t MAX_HEAD_DIM = 512;           // eight columns to a lane

int64_t up128(int64_t n) { return (n + 127) / 128 * 128; }

int check_product_sizes(const mega_moe_product_args* a) {
    if (!a) return bad("the argument block is NULL");
    if (a->m < 0 || a->m > MAX_TOKENS) return fail(MEGA_MOE_ERR_INVALID_ARG, "m must be in [0, %d], got %d", MAX_TOKENS, a->m);
    if (a->n < 0 || a->n > MAX_TOKENS || a->n % 8)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "n must be a multiple of 8 in [0, %d], got %d", MAX_TOKENS, a->n);
    if (a->k < 0 || a->k > MAX_TOKENS || a->k % 128)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "k must be a multiple of 128 in [0, %d], got %d", MAX_TOKENS, a->k);
    if (a->b_scale != MEGA_MOE_SCALE_BLOCK && a->b_scale != MEGA_MOE_SCALE_ROW) return bad("unknown b_scale");
    if (!type_ok(a->out_type)) return bad("out_type is neither MEGA_MOE_BF16 nor MEGA_MOE_F32");
    if (a->reserved != 0) return bad("reserved must be 0");
    return MEGA_MOE_OK;
}

// What mega_moe_quantize and mega_moe_swiglu_backward check alike.
template <typename Args>
int check_quantize(const Args& a) {
    if (const int rc = check_tokens(a.num_tokens)) return rc;
    if (a.columns < 128 || a.columns > MAX_COLUMNS || a.columns % 128)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "columns must be a multiple of 128 in [128, %d], got %d", MAX_COLUMNS, a.columns);
    if (!type_ok(a.x_type)) return bad("x_type is neither MEGA_MOE_BF16 nor MEGA_MOE_F32");
    if (!(a.activation_clamp >= 0.0f)) return bad("activation_clamp must be >= 0");
    if ((a.q == nullptr) != (a.q_sf == nullptr) || (a.qt == nullptr) != (a.qt_sf == nullptr))
        return bad("q and q_sf, and qt and qt_sf, go together");
    return MEGA_MOE_OK;
}

template <typename Args>
int check_rotary(const Args& a) {
    if (const int rc = check_tokens(a.num_tokens)) return rc;
    if (a.q_heads < 0 || a.q_heads > MAX_HEADS || a.k_heads < 0 || a.k_heads > MAX_HEADS || a.q_heads + a.k_heads == 0)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "q_heads and k_heads must be in [0, %d], and not both 0", MAX_HEADS);
    if (a.head_dim < 8 || a.head_dim % 8) return fail(MEGA_MOE_ERR_INVALID_ARG, "head_dim must be a positive multiple of 8, got %d", a.head_dim);
    if (a.head_dim > MAX_HEAD_DIM) return fail(MEGA_MOE_ERR_UNSUPPORTED, "built for head_dim <= %d, got %d", MAX_HEAD_DIM, a.head_dim);
    if (a.rotary_dim < 0 || a.rotary_dim % 16 || a.rotary_dim > a.head_dim)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "rotary_dim must be a multiple of 16 in [0, head_dim], got %d", a.rotary_dim);
    if (a.rotary_start < 0 || a.rotary_start % 8 || a.rotary_start > a.head_dim - a.rotary_dim)
        return bad("rotary_start must be a multiple of 8, with the rotated columns inside the head");
    if (a.layout != MEGA_MOE_ROTARY_HALF && a.layout != MEGA_MOE_ROTARY_INTERLEAVED) return bad("unknown layout");
    if (!type_ok(a.type) || !type_ok(a.weight_type)) return bad("a type is neither MEGA_MOE_BF16 nor MEGA_MOE_F32");
    if (a.first_position < 0 || (int64_t)a.first_position + a.num_tokens > (int64_t)INT32_MAX + 1)
        return bad("first_position must be >= 0, and the last position a 32-bit number");
    if (!(a.eps >= 0.0f) || std::isinf(a.eps)) return bad("eps must be finite and >= 0");
    if (!std::isfinite(a.scale)) return bad("scale must be finite");
    if ((a.q_weight && a.q_heads == 0) || (a.k_weight && a.k_heads == 0)) return bad("a weight needs its heads");
    return MEGA_MOE_OK;
}

// The strides of one tensor of heads, resolved; false if they cannot be used.
// Dense rows of one head after another where they are 0.  Those of no heads are of no matter.
bool head_strides(int64_t& token, int64_t& head, int heads, int D) {
    if (heads == 0) return true;
    if (head == 0) head = D;
    if (head < D || head % 8 || head > MAX_HEAD_STRIDE) return false;
    const int64_t row = (heads - 1) * head + D;
    if (token == 0) token = head * heads;
    return token >= row && token % 8 == 0 && token <= ((int64_t)1 << 38);
}

void add_heads(Tensors& ts, const char* name, const void* p, int64_t T, int heads, int D, int64_t token, int64_t head, int64_t size, bool out) {
    if (heads > 0) ts.add_parts(name, p, T, heads, D, head, token, size, out);
}

int64_t rotary_bytes(const mega_moe_rotary_backward_args& a) {
    return (int64_t)rotary_backward_blocks(a) * rotary_sums(a) * a.head_dim * 4;
}

int check_rotary_backward(const mega_moe_rotary_backward_args* a) {
    if (!a) return bad("the argument block is NULL");
    if (const int rc = check_rotary(*a)) return rc;
    if ((a->dq_weight && !a->q_weight) || (a->dk_weight && !a->k_weight)) return bad("a weight's gradient needs the weight");
    return MEGA_MOE_OK;
}

}  // namespace

extern "C" {

int64_t mega_moe_product_workspace_bytes(const mega_moe_product_args* a) {
    if (check_product_sizes(a)) return -1;
    return a->m == 0 || a->n == 0 ? 0 : product_workspace(product_plan(a->m, a->n, a->k, a->out_type), a->m, a->n);
}

int mega_moe_product(const mega_moe_product_args* args, void* stream) {
    int rc = check_product_sizes(args);
    if (rc) return rc;
    mega_moe_product_args a = *args;
    if (a.m == 0 || a.n == 0) return ok();
    if (!a.out) return bad("out is NULL");
    if (a.k > 0 && (!a.a || !a.a_sf || !a.b || !a.b_sf)) return bad("a, a_sf, b or b_sf is NULL");
    if (!lines_aligned({a.a, a.b, a.add, a.out}) || !words_aligned({a.a_sf, a.b_sf}))
        return bad("a, b, add and out must be 16-byte aligned, the scales 4-byte");
    const int64_t m = a.m, n = a.n, k = a.k, blocks = k / 128;
    const int64_t b_rows = a.b_scale == MEGA_MOE_SCALE_ROW ? n : up128(n) / 128;
    a.a_stride = stride_of(a.a_stride, k, 16);
    a.b_stride = stride_of(a.b_stride, k, 16);
    a.a_sf_stride = stride_of(a.a_sf_stride, blocks, 1);
    a.b_sf_stride = stride_of(a.b_sf_stride, blocks, 1);
    a.add_stride = stride_of(a.add_stride, n, 8);
    a.out_stride = stride_of(a.out_stride, n, 8);
    if (a.a_stride < 0 || a.b_stride < 0 || a.a_sf_stride < 0 || a.b_sf_stride < 0 || a.add_stride < 0 || a.out_stride < 0)
        return bad("a stride is shorter than its row, or not a multiple of 16 (codes) or 8 (add and out)");
    if (a.a_stride > MAX_X_STRIDE || a.b_stride > MAX_X_STRIDE || a.a_sf_stride > MAX_SF_STRIDE || a.b_sf_stride > MAX_SF_STRIDE)
        return fail(MEGA_MOE_ERR_UNSUPPORTED, "built for strides of codes <= %lld and of scales <= %lld",
                    (long long)MAX_X_STRIDE, (long long)MAX_SF_STRIDE);
    const ProductPlan plan = product_plan(a.m, a.n, a.k, a.out_type);
    const int64_t need = product_workspace(plan, a.m, a.n), size = type_bytes(a.out_type);
    if ((rc = check_workspace(a.workspace, a.workspace_bytes, need))) return rc;
    Tensors ts;
    if (k > 0) {
        ts.add("a", a.a, m, k, a.a_stride, 1, false);
        ts.add("a_sf", a.a_sf, m, blocks, a.a_sf_stride, 4, false);
        ts.add("b", a.b, n, k, a.b_stride, 1, false);
        ts.add("b_sf", a.b_sf, b_rows, blocks, a.b_sf_stride, 4, false);
    }
    ts.add("add", a.add, m, n, a.add_stride, size, false);
    ts.add("out", a.out, m, n, a.out_stride, size, true);
    ts.add("workspace", a.workspace, 1, need, need, 1, true);
    if ((rc = ts.check("out", "add")) || (rc = check_device(k > 0 ? (const void*)a.a : a.out, stream))) return rc;
    launch_product(a, plan, (hipStream_t)stream);
    return launched();
}

int mega_moe_quantize(const mega_moe_quantize_args* args, void* stream) {
    if (!args) return bad("the argument block is NULL");
    mega_moe_quantize_args a = *args;
    int rc = check_quantize(a);
    if (rc) return rc;
    if (a.activation != MEGA_MOE_ACT_NONE && a.activation != MEGA_MOE_ACT_SWIGLU) return bad("unknown activation");
    if (a.scale != MEGA_MOE_SCALE_BLOCK && a.scale != MEGA_MOE_SCALE_ROW) return bad("unknown scale");
    const bool swiglu = a.activation == MEGA_MOE_ACT_SWIGLU;
    if (!swiglu && (a.up || a.activation_clamp != 0.0f)) return bad("up and activation_clamp need MEGA_MOE_ACT_SWIGLU");
    if (!a.h && !a.q && !a.qt) return bad("no output: h, q and qt are NULL");
    if (a.num_tokens == 0) return ok();
    if (!a.x || (swiglu && !a.up)) return bad("x or up is NULL");
    if (!lines_aligned({a.x, a.up, a.h, a.q, a.qt}) || !words_aligned({a.q_sf, a.qt_sf}))
        return bad("the tensors must be 16-byte aligned, the scales 4-byte");
    const int64_t T = a.num_tokens, C = a.columns, Tp = up128(T);
    for (int64_t* s : {&a.x_stride, &a.up_stride, &a.h_stride})
        if ((*s = stride_of(*s, C, 8)) < 0) return bad("a stride is shorter than its row, or not a multiple of 8");
    const bool block = a.scale == MEGA_MOE_SCALE_BLOCK;
    const int64_t size = type_bytes(a.x_type);
    Tensors ts;
    ts.add("x", a.x, T, C, a.x_stride, size, false);
    ts.add("up", a.up, T, C, a.up_stride, size, false);
    ts.add("h", a.h, T, C, a.h_stride, 2, true);
    ts.add("q", a.q, T, C, C, 1, true);
    ts.add("q_sf", a.q_sf, block ? Tp / 128 : T, C / 128, C / 128, 4, true);
    ts.add("qt", a.qt, C, Tp, Tp, 1, true);
    ts.add("qt_sf", a.qt_sf, block ? C / 128 : C, Tp / 128, Tp / 128, 4, true);
    if ((rc = ts.check()) || (rc = check_device(a.x, stream))) return rc;
    launch_quantize(a, (hipStream_t)stream);
    return launched();
}

int mega_moe_swiglu_backward(const mega_moe_swiglu_backward_args* args, void* stream) {
    if (!args) return bad("the argument block is NULL");
    mega_moe_swiglu_backward_args a = *args;
    int rc = check_quantize(a);
    if (rc) return rc;
    if (!a.dx && !a.dup && !a.q && !a.qt) return bad("no output: dx, dup, q and qt are NULL");
    if (a.num_tokens == 0) return ok();
    if (!a.x || !a.up || !a.dh) return bad("x, up or dh is NULL");
    if (!lines_aligned({a.x, a.up, a.dh, a.dx, a.dup, a.q, a.qt}) || !words_aligned({a.q_sf, a.qt_sf}))
        return bad("the tensors must be 16-byte aligned, the scales 4-byte");
    const int64_t T = a.num_tokens, C = a.columns, Tp = up128(T), size = type_bytes(a.x_type);
    for (int64_t* s : {&a.x_stride, &a.up_stride, &a.dh_stride, &a.dx_stride, &a.dup_stride})
        if ((*s = stride_of(*s, C, 8)) < 0) return bad("a stride is shorter than its row, or not a multiple of 8");
    Tensors ts;
    ts.add("x", a.x, T, C, a.x_stride, size, false);
    ts.add("up", a.up, T, C, a.up_stride, size, false);
    ts.add("dh", a.dh, T, C, a.dh_stride, size, false);
    ts.add("dx", a.dx, T, C, a.dx_stride, size, true);
    ts.add("dup", a.dup, T, C, a.dup_stride, size, true);
    ts.add("q", a.q, T, 2 * C, 2 * C, 1, true);
    ts.add("q_sf", a.q_sf, T, C / 64, C / 64, 4, true);
    ts.add("qt", a.qt, 2 * C, Tp, Tp, 1, true);
    ts.add("qt_sf", a.qt_sf, 2 * C, Tp / 128, Tp / 128, 4, true);
    if ((rc = ts.check()) || (rc = check_device(a.x, stream))) return rc;
    launch_swiglu_backward(a, (hipStream_t)stream);
    return launched();
}

int mega_moe_rotary(const mega_moe_rotary_args* args, void* stream) {
    if (!args) return bad("the argument block is NULL");
    mega_moe_rotary_args a = *args;
    int rc = check_rotary(a);
    if (rc) return rc;
    if (a.num_tokens == 0) return ok();
    if ((a.q_heads > 0 && (!a.q || !a.q_out)) || (a.k_heads > 0 && (!a.k || !a.k_out))) return bad("q, k, q_out or k_out is NULL");
    if (a.rotary_dim > 0 && !a.inv_freq) return bad("inv_freq is NULL");
    if (!lines_aligned({a.q, a.k, a.q_weight, a.k_weight, a.q_out, a.k_out}) || !words_aligned({a.positions, a.inv_freq}))
        return bad("the tensors of heads and the weights must be 16-byte aligned, positions and inv_freq 4-byte");
    const int D = a.head_dim;
    if (!head_strides(a.q_stride, a.q_head_stride, a.q_heads, D) || !head_strides(a.k_stride, a.k_head_stride, a.k_heads, D) ||
        !head_strides(a.q_out_stride, a.q_out_head_stride, a.q_heads, D) ||
        !head_strides(a.k_out_stride, a.k_out_head_stride, a.k_heads, D))
        return bad("a stride is shorter than its row or head, too long, or not a multiple of 8");
    const int64_t T = a.num_tokens, size = type_bytes(a.type), ws = type_bytes(a.weight_type);
    if (a.q_heads > 0 && a.q_out == a.q && (a.q_out_stride != a.q_stride || a.q_out_head_stride != a.q_head_stride))
        return bad("q_out may be q only with the same strides");
    if (a.k_heads > 0 && a.k_out == a.k && (a.k_out_stride != a.k_stride || a.k_out_head_stride != a.k_head_stride))
        return bad("k_out may be k only with the same strides");
    Tensors ts;
    add_heads(ts, "q", a.q, T, a.q_heads, D, a.q_stride, a.q_head_stride, size, false);
    add_heads(ts, "k", a.k, T, a.k_heads, D, a.k_stride, a.k_head_stride, size, false);
    ts.add("q_weight", a.q_weight, 1, D, D, ws, false);
    ts.add("k_weight", a.k_weight, 1, D, D, ws, false);
    ts.add("positions", a.positions, 1, T, T, 4, false);
    ts.add("inv_freq", a.inv_freq, 1, a.rotary_dim / 2, a.rotary_dim / 2, 4, false);
    add_heads(ts, "q_out", a.q_out, T, a.q_heads, D, a.q_out_stride, a.q_out_head_stride, size, true);
    add_heads(ts, "k_out", a.k_out, T, a.k_heads, D, a.k_out_stride, a.k_out_head_stride, size, true);
    if ((rc = ts.check("q_out", "q", "k_out", "k")) || (rc = check_device(a.q_heads > 0 ? a.q : a.k, stream))) return rc;
    launch_rotary(a, (hipStream_t)stream);
    return launched();
}

int64_t mega_moe_rotary_workspace_bytes(const mega_moe_rotary_backward_args* a) {
    if (check_rotary_backward(a)) return -1;
    return rotary_bytes(*a);
}

int mega_moe_rotary_backward(const mega_moe_rotary_backward_args* args, void* stream) {
    int rc = check_rotary_backward(args);
    if (rc) return rc;
    mega_moe_rotary_backward_args a = *args;
    if (a.num_tokens == 0 && rotary_sums(a) == 0) return ok();
    if (a.num_tokens > 0) {
        if ((a.q_heads > 0 && (!a.dq_out || !a.dq)) || (a.k_heads > 0 && (!a.dk_out || !a.dk)))
            return bad("dq_out, dk_out, dq or dk is NULL");
        if ((a.q_weight && !a.q) || (a.k_weight && !a.k)) return bad("a weight needs its q or k");
        if (a.rotary_dim > 0 && !a.inv_freq) return bad("inv_freq is NULL");
    }
    if (!lines_aligned({a.q, a.k, a.q_weight, a.k_weight, a.dq_out, a.dk_out, a.dq, a.dk}) ||
        !words_aligned({a.positions, a.inv_freq, a.dq_weight, a.dk_weight}))
        return bad("the tensors of heads and the weights must be 16-byte aligned, the other arrays 4-byte");
    const int D = a.head_dim;
    if (!head_strides(a.q_stride, a.q_head_stride, a.q_heads, D) || !head_strides(a.k_stride, a.k_head_stride, a.k_heads, D) ||
        !head_strides(a.dq_out_stride, a.dq_out_head_stride, a.q_heads, D) ||
        !head_strides(a.dk_out_stride, a.dk_out_head_stride, a.k_heads, D) ||
        !head_strides(a.dq_stride, a.dq_head_stride, a.q_heads, D) || !head_strides(a.dk_stride, a.dk_head_stride, a.k_heads, D))
        return bad("a stride is shorter than its row or head, too long, or not a multiple of 8");
    if (a.q_heads > 0 && a.dq && a.dq == a.dq_out && (a.dq_stride != a.dq_out_stride || a.dq_head_stride != a.dq_out_head_stride))
        return bad("dq may be dq_out only with the same strides");
    if (a.k_heads > 0 && a.dk && a.dk == a.dk_out && (a.dk_stride != a.dk_out_stride || a.dk_head_stride != a.dk_out_head_stride))
        return bad("dk may be dk_out only with the same strides");
    const int64_t need = rotary_bytes(a);
    if ((rc = check_workspace(a.workspace, a.workspace_bytes, need))) return rc;
    const int64_t T = a.num_tokens, size = type_bytes(a.type), ws = type_bytes(a.weight_type);
    Tensors ts;
    if (a.q_weight) add_heads(ts, "q", a.q, T, a.q_heads, D, a.q_stride, a.q_head_stride, size, false);
    if (a.k_weight) add_heads(ts, "k", a.k, T, a.k_heads, D, a.k_stride, a.k_head_stride, size, false);
    ts.add("q_weight", a.q_weight, 1, D, D, ws, false);
    ts.add("k_weight", a.k_weight, 1, D, D, ws, false);
    ts.add("positions", a.positions, 1, T, T, 4, false);
    ts.add("inv_freq", a.inv_freq, 1, a.rotary_dim / 2, a.rotary_dim / 2, 4, false);
    add_heads(ts, "dq_out", a.dq_out, T, a.q_heads, D, a.dq_out_stride, a.dq_out_head_stride, size, false);
    add_heads(ts, "dk_out", a.dk_out, T, a.k_heads, D, a.dk_out_stride, a.dk_out_head_stride, size, false);
    add_heads(ts, "dq", a.dq, T, a.q_heads, D, a.dq_stride, a.dq_head_stride, size, true);
    add_heads(ts, "dk", a.dk, T, a.k_heads, D, a.dk_stride, a.dk_head_stride, size, true);
    ts.add("dq_weight", a.dq_weight, 1, D, D, 4, true);
    ts.add("dk_weight", a.dk_weight, 1, D, D, 4, true);
    ts.add("workspace", a.workspace, 1, need, need, 1, true);
    if ((rc = ts.check("dq", "dq_out", "dk", "dk_out"))) return rc;
    const void* first = a.num_tokens > 0 ? (a.q_heads > 0 ? a.dq_out : a.dk_out) : a.dq_weight ? a.dq_weight : a.dk_weight;
    if ((rc = check_device(first, stream))) return rc;
    launch_rotary_backward(a, (hipStream_t)stream);
    return launched();
}

int mega_moe_rotary_frequencies(const mega_moe_rotary_frequencies_args* a) {
    if (!a) return bad("the argument block is NULL");
    if (a->rotary_dim < 16 || a->rotary_dim % 16 || a->rotary_dim > MAX_HEAD_DIM)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "rotary_dim must be a multiple of 16 in [16, %d], got %d", MAX_HEAD_DIM, a->rotary_dim);
    if (a->scaling < MEGA_MOE_ROTARY_PLAIN || a->scaling > MEGA_MOE_ROTARY_BY_PARTS) return bad("unknown scaling");
    if (!(a->base > 1.0) || !std::isfinite(a->base)) return bad("base must be finite and > 1");
    if (a->scaling == MEGA_MOE_ROTARY_PLAIN ? a->factor != 0.0 : !(a->factor >= 1.0) || !std::isfinite(a->factor))
        return bad("factor must be finite and >= 1 (0 without scaling)");
    const bool parts = a->scaling == MEGA_MOE_ROTARY_BY_PARTS;
    if (parts && (!(a->original_length > 0.0) || !std::isfinite(a->original_length) || !(a->slow_turns > 0.0) ||
                  !(a->fast_turns > a->slow_turns) || !std::isfinite(a->fast_turns)))
        return bad("original_length and slow_turns must be > 0 and fast_turns > slow_turns, all finite");
    if (!a->inv_freq) return bad("inv_freq is NULL");
    const int half = a->rotary_dim / 2;
    double lo = 0.0, hi = 0.0;
    if (parts) {
        // the index whose frequency makes `turns` turns over the original length
        const auto index = [&](double turns) {
            return a->rotary_dim * std::log(a->original_length / (turns * 6.283185307179586)) / (2.0 * std::log(a->base));
        };
        lo = std::fmax(std::floor(index(a->fast_turns)), 0.0);
        hi = std::fmin(std::ceil(index(a->slow_turns)), a->rotary_dim - 1.0);    // the last frequency may lie between both
        lo = std::fmin(lo, hi - 1.0);                   // all of them are slow, or all fast
    }
    for (int i = 0; i < half; ++i) {
        double f = std::pow(a->base, -2.0 * i / a->rotary_dim);
        if (a->scaling == MEGA_MOE_ROTARY_LINEAR) f /= a->factor;
        if (parts) {
            const double slow = std::fmin(std::fmax((i - lo) / (hi - lo), 0.0), 1.0);
            f = f / a->factor * slow + f * (1.0 - slow);
        }
        a->inv_freq[i] = (float)f;
    }
    if (a->scale) *a->scale = parts ? (float)(0.1 * std::log(a->factor) + 1.0) : 1.0f;
    return ok();
}

}  // extern "C"
