// Host side of the operators around the layer (the second half of
// include/mega_moe.h): argument checks and launches.
#include <hip/hip_runtime.h>

#include <cmath>

#include "checks.h"
#include "mega_moe.h"
#include "moe_args.h"
#include "norm.h"
#include "router.h"
#include "router_logits.h"

using namespace mega_moe;

namespace {

constexpr int32_t MAX_HIDDEN = 8192;        // as the layer

int check_hidden(int32_t h) {
    if (h < 8 || h % 8) return fail(MEGA_MOE_ERR_INVALID_ARG, "hidden must be a positive multiple of 8, got %d", h);
    if (h > MAX_HIDDEN) return fail(MEGA_MOE_ERR_UNSUPPORTED, "built for hidden <= %d, got %d", MAX_HIDDEN, h);
    return MEGA_MOE_OK;
}

// What mega_moe_norm and its gradient check alike.
template <typename Args>
int check_norm(const Args& a, bool q) {
    if (const int rc = check_tokens(a.num_tokens)) return rc;
    if (const int rc = check_hidden(a.hidden)) return rc;
    if (q && a.hidden % 128) return bad("q needs hidden to be a multiple of 128");
    if (!type_ok(a.stream_type) || !type_ok(a.weight_type) || !type_ok(a.gate_type))
        return bad("a type is neither MEGA_MOE_BF16 nor MEGA_MOE_F32");
    if (a.gate_kind < MEGA_MOE_GATE_NONE || a.gate_kind > MEGA_MOE_GATE_FULL) return bad("unknown gate_kind");
    if (a.reserved != 0) return bad("reserved must be 0");
    if (!(a.post_eps >= 0.0f) || !(a.pre_eps >= 0.0f) || std::isinf(a.post_eps) || std::isinf(a.pre_eps))
        return bad("post_eps and pre_eps must be finite and >= 0");
    if (!std::isfinite(a.residual_scale)) return bad("residual_scale must be finite");
    if (!a.y && (a.gate_kind != MEGA_MOE_GATE_NONE || a.gate || a.post_weight || a.residual_scale != 1.0f))
        return bad("a gate, post_weight and residual_scale other than 1 need y");
    if ((a.gate_kind == MEGA_MOE_GATE_NONE) != (a.gate == nullptr)) return bad("gate and gate_kind do not go together");
    return MEGA_MOE_OK;
}

// What the norms' tensors must be: aligned to 16 bytes, but for a [T] gate.
template <typename Args>
int check_norm_gate(const Args& a) {
    if (a.gate_kind == MEGA_MOE_GATE_TOKEN ? !aligned(a.gate, type_bytes(a.gate_type)) : !aligned(a.gate, 16))
        return bad("gate is not aligned");
    return MEGA_MOE_OK;
}

template <typename Args>
void add_norm_inputs(Tensors& ts, const Args& a) {
    const int64_t T = a.num_tokens, H = a.hidden;
    ts.add("y", a.y, T, H, a.y_stride, 2, false);
    if (a.gate_kind == MEGA_MOE_GATE_TOKEN) ts.add("gate", a.gate, 1, T, T, type_bytes(a.gate_type), false);
    else if (a.gate_kind == MEGA_MOE_GATE_CHANNEL) ts.add("gate", a.gate, 1, H, H, type_bytes(a.gate_type), false);
    else ts.add("gate", a.gate, T, H, a.gate_stride, type_bytes(a.gate_type), false);
    ts.add("post_weight", a.post_weight, 1, H, H, type_bytes(a.weight_type), false);
    ts.add("pre_weight", a.pre_weight, 1, H, H, type_bytes(a.weight_type), false);
}

int check_norm_backward(const mega_moe_norm_backward_args& a) {
    const int rc = check_norm(a, false);
    if (rc) return rc;
    if ((a.dn || a.dpre_weight) && !a.pre_weight) return bad("dn and dpre_weight need pre_weight");
    if (a.dy && !a.y) return bad("dy needs y");
    if (a.dgate && !a.gate) return bad("dgate needs the gate");
    if (a.dpost_weight && !a.post_weight) return bad("dpost_weight needs post_weight");
    return MEGA_MOE_OK;
}

int64_t norm_backward_bytes(const mega_moe_norm_backward_args& a) {
    return (int64_t)norm_backward_blocks(a.num_tokens, a.hidden) * norm_sums(a) * a.hidden * 4;
}

int check_logits_sizes(const mega_moe_router_logits_args* a) {
    if (!a) return bad("the argument block is NULL");
    if (const int rc = check_tokens(a->num_tokens)) return rc;
    if (const int rc = check_hidden(a->hidden)) return rc;
    if (a->num_experts < 1 || a->num_experts > MAX_EXPERTS)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "num_experts must be in [1, %d], got %d", MAX_EXPERTS, a->num_experts);
    if (!type_ok(a->weight_type)) return bad("weight_type is neither MEGA_MOE_BF16 nor MEGA_MOE_F32");
    return MEGA_MOE_OK;
}

// The row strides of a router product, resolved into `a`.
int logits_strides(mega_moe_router_logits_args& a) {
    a.x_stride = stride_of(a.x_stride, a.hidden, 8);
    a.dx_add_stride = stride_of(a.dx_add_stride, a.hidden, 8);
    a.dx_stride = stride_of(a.dx_stride, a.hidden, 8);
    a.logits_stride = stride_of(a.logits_stride, a.num_experts, 1);
    a.dlogits_stride = stride_of(a.dlogits_stride, a.num_experts, 1);
    if (a.x_stride > MAX_X_STRIDE)
        return fail(MEGA_MOE_ERR_UNSUPPORTED, "built for x_stride <= %lld", (long long)MAX_X_STRIDE);
    if (a.x_stride < 0 || a.dx_add_stride < 0 || a.dx_stride < 0 || a.logits_stride < 0 || a.dlogits_stride < 0)
        return bad("a stride is shorter than its row, or not a multiple of 8");
    return MEGA_MOE_OK;
}

// What the calls on logits check alike.
template <typename Args>
int check_router(const Args& a) {
    if (const int rc = check_tokens(a.num_tokens)) return rc;
    if (a.num_experts < 1 || a.num_experts > MAX_EXPERTS)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "num_experts must be in [1, %d], got %d", MAX_EXPERTS, a.num_experts);
    if (a.num_topk < 1 || a.num_topk > MAX_EXPERTS)
        return fail(MEGA_MOE_ERR_INVALID_ARG, "num_topk must be in [1, %d], got %d", MAX_EXPERTS, a.num_topk);
    if (!type_ok(a.logits_type)) return bad("logits_type is neither MEGA_MOE_BF16 nor MEGA_MOE_F32");
    if (a.score != MEGA_MOE_SCORE_SOFTMAX && a.score != MEGA_MOE_SCORE_SIGMOID) return bad("unknown score");
    return MEGA_MOE_OK;
}

template <typename Args>
int check_sequences(const Args& a) {
    if (a.num_sequences < 0 || (a.num_sequences > 1 && !a.cu_seqlens)) return bad("num_sequences needs cu_seqlens");
    if (a.cu_seqlens && a.num_sequences < 1) return bad("cu_seqlens needs num_sequences");
    if (a.num_sequences > MAX_TOKENS) return fail(MEGA_MOE_ERR_INVALID_ARG, "num_sequences must be at most %d", MAX_TOKENS);
    if (!std::isfinite(a.balance_coeff) || !std::isfinite(a.z_coeff)) return bad("the coefficients must be finite");
    return MEGA_MOE_OK;
}

int check_balance_sizes(const mega_moe_balance_loss_args* a) {
    if (!a) return bad("the argument block is NULL");
    if (const int rc = check_router(*a)) return rc;
    if (const int rc = check_sequences(*a)) return rc;
    const int64_t groups = balance_finish_groups(a->num_sequences, a->num_experts);
    if (groups > BALANCE_MAX_GROUPS)
        return fail(MEGA_MOE_ERR_UNSUPPORTED, "built for num_sequences * ceil(num_experts / 32) <= %lld, got %lld",
                    (long long)BALANCE_MAX_GROUPS, (long long)groups);
    return MEGA_MOE_OK;
}

}  // namespace

extern "C" {

int mega_moe_norm(const mega_moe_norm_args* args, void* stream) {
    if (!args) return bad("the argument block is NULL");
    mega_moe_norm_args a = *args;
    int rc = check_norm(a, a.q != nullptr);
    if (rc) return rc;
    if ((a.q == nullptr) != (a.q_sf == nullptr)) return bad("q and q_sf go together");
    if ((a.n || a.q) && !a.pre_weight) return bad("n and q need pre_weight");
    if (!a.r && !a.n && !a.q) return bad("no output: r, n and q are NULL");
    if (a.num_tokens == 0) return ok();
    if (!a.h) return bad("h is NULL");
    if (!lines_aligned({a.h, a.y, a.post_weight, a.pre_weight, a.r, a.n, a.q}) || !words_aligned({a.q_sf}))
        return bad("the tensors of H columns must be 16-byte aligned, q_sf 4-byte");
    if ((rc = check_norm_gate(a))) return rc;
    const int64_t T = a.num_tokens, H = a.hidden;
    a.h_stride = stride_of(a.h_stride, H, 8);
    a.y_stride = stride_of(a.y_stride, H, 8);
    a.gate_stride = stride_of(a.gate_stride, H, 8);
    a.r_stride = stride_of(a.r_stride, H, 8);
    a.n_stride = stride_of(a.n_stride, H, 8);
    if (a.h_stride < 0 || a.y_stride < 0 || a.gate_stride < 0 || a.r_stride < 0 || a.n_stride < 0)
        return bad("a stride is shorter than its row, or not a multiple of 8");
    Tensors ts;
    ts.add("h", a.h, T, H, a.h_stride, type_bytes(a.stream_type), false);
    add_norm_inputs(ts, a);
    ts.add("r", a.r, T, H, a.r_stride, type_bytes(a.stream_type), true);
    ts.add("n", a.n, T, H, a.n_stride, 2, true);
    ts.add("q", a.q, T, H, H, 1, true);
    ts.add("q_sf", a.q_sf, T, H / 128, H / 128, 4, true);
    if ((rc = ts.check("r", "h"))) return rc;
    if (!a.n && !a.q) a.pre_weight = nullptr;      // nothing to norm for
    if ((rc = check_device(a.h, stream))) return rc;
    launch_norm(a, (hipStream_t)stream);
    return launched();
}

int64_t mega_moe_norm_workspace_bytes(const mega_moe_norm_backward_args* a) {
    if (!a) return bad("the argument block is NULL");
    if (check_norm_backward(*a)) return -1;
    return norm_backward_bytes(*a);
}

int mega_moe_norm_backward(const mega_moe_norm_backward_args* args, void* stream) {
    if (!args) return bad("the argument block is NULL");
    mega_moe_norm_backward_args a = *args;
    int rc = check_norm_backward(a);
    if (rc) return rc;
    if (!a.dh && !a.dy && !a.dgate && !a.dpost_weight && !a.dpre_weight) return bad("no output: every gradient is NULL");
    if (a.num_tokens == 0 && norm_sums(a) == 0) return ok();
    if (a.num_tokens > 0) {
        if (!a.dr && !a.dn) return bad("dr and dn are both NULL");
        if (a.dn && !a.r) return bad("dn needs r");
    }
    if (!lines_aligned({a.r, a.y, a.post_weight, a.pre_weight, a.dr, a.dn, a.dh, a.dy, a.dpost_weight, a.dpre_weight}))
        return bad("the tensors of H columns must be 16-byte aligned");
    if ((rc = check_norm_gate(a))) return rc;
    if (a.gate_kind == MEGA_MOE_GATE_TOKEN ? !aligned(a.dgate, 4) : !aligned(a.dgate, 16))
        return bad("dgate is not aligned");
    const int64_t T = a.num_tokens, H = a.hidden;
    int64_t* strides[] = {&a.r_stride, &a.y_stride, &a.gate_stride, &a.dr_stride,
                          &a.dn_stride, &a.dh_stride, &a.dy_stride, &a.dgate_stride};
    for (int64_t* s : strides)
        if ((*s = stride_of(*s, H, 8)) < 0) return bad("a stride is shorter than its row, or not a multiple of 8");
    const int64_t need = norm_backward_bytes(a);
    if ((rc = check_workspace(a.workspace, a.workspace_bytes, need))) return rc;
    const int64_t sb = type_bytes(a.stream_type);
    Tensors ts;
    ts.add("r", a.r, T, H, a.r_stride, sb, false);
    add_norm_inputs(ts, a);
    ts.add("dr", a.dr, T, H, a.dr_stride, sb, false);
    ts.add("dn", a.dn, T, H, a.dn_stride, 2, false);
    ts.add("dh", a.dh, T, H, a.dh_stride, sb, true);
    ts.add("dy", a.dy, T, H, a.dy_stride, 2, true);
    if (a.gate_kind == MEGA_MOE_GATE_TOKEN) ts.add("dgate", a.dgate, 1, T, T, 4, true);
    else if (a.gate_kind == MEGA_MOE_GATE_CHANNEL) ts.add("dgate", a.dgate, 1, H, H, 4, true);
    else ts.add("dgate", a.dgate, T, H, a.dgate_stride, type_bytes(a.gate_type), true);
    ts.add("dpost_weight", a.dpost_weight, 1, H, H, 4, true);
    ts.add("dpre_weight", a.dpre_weight, 1, H, H, 4, true);
    ts.add("workspace", a.workspace, 1, need, need, 1, true);
    if ((rc = ts.check("dh", "dr"))) return rc;
    const void* first = T > 0 ? (a.dr ? a.dr : a.dn) : a.dpre_weight ? a.dpre_weight : a.dpost_weight ? a.dpost_weight : a.dgate;
    if ((rc = check_device(first, stream))) return rc;
    launch_norm_backward(a, (hipStream_t)stream);
    return launched();
}

int64_t mega_moe_router_logits_workspace_bytes(const mega_moe_router_logits_args* a) {
    if (check_logits_sizes(a)) return -1;
    return router_logits_workspace(*a);
}

int mega_moe_router_logits(const mega_moe_router_logits_args* args, void* stream) {
    int rc = check_logits_sizes(args);
    if (rc) return rc;
    mega_moe_router_logits_args a = *args;
    if (a.num_tokens == 0) return ok();
    if (!a.x || !a.w || !a.logits) return bad("x, w or logits is NULL");
    if (!lines_aligned({a.x, a.w}) || !words_aligned({a.logits}))
        return bad("x and w must be 16-byte aligned, logits 4-byte");
    if ((rc = logits_strides(a))) return rc;
    const int64_t T = a.num_tokens, H = a.hidden, E = a.num_experts, need = router_logits_workspace(a);
    if ((rc = check_workspace(a.workspace, a.workspace_bytes, need))) return rc;
    Tensors ts;
    ts.add("x", a.x, T, H, a.x_stride, 2, false);
    ts.add("w", a.w, E, H, H, type_bytes(a.weight_type), false);
    ts.add("logits", a.logits, T, E, a.logits_stride, 4, true);
    ts.add("workspace", a.workspace, 1, need, need, 1, true);
    if ((rc = ts.check()) || (rc = check_device(a.x, stream))) return rc;
    launch_router_logits(a, (hipStream_t)stream);
    return launched();
}

int mega_moe_router_logits_backward(const mega_moe_router_logits_args* args, void* stream) {
    int rc = check_logits_sizes(args);
    if (rc) return rc;
    mega_moe_router_logits_args a = *args;
    if (!a.dx && !a.dw) return bad("no output: dx and dw are NULL");
    if (a.dx_add && !a.dx) return bad("dx_add needs dx");
    if (a.num_tokens == 0) {
        a.dx = nullptr;
        if (!a.dw) return ok();
    } else {
        if (!a.dlogits) return bad("dlogits is NULL");
        if (a.dx && !a.w) return bad("dx needs w");
        if (a.dw && !a.x) return bad("dw needs x");
    }
    if (!lines_aligned({a.x, a.w, a.dx_add, a.dx, a.dw}) || !words_aligned({a.dlogits}))
        return bad("x, w, dx_add, dx and dw must be 16-byte aligned, dlogits 4-byte");
    if ((rc = logits_strides(a))) return rc;
    const int64_t T = a.num_tokens, H = a.hidden, E = a.num_experts, need = router_logits_workspace(a);
    if ((rc = check_workspace(a.workspace, a.workspace_bytes, need))) return rc;
    Tensors ts;
    ts.add("x", a.x, T, H, a.x_stride, 2, false);
    ts.add("w", a.w, E, H, H, type_bytes(a.weight_type), false);
    ts.add("dlogits", a.dlogits, T, E, a.dlogits_stride, 4, false);
    ts.add("dx_add", a.dx_add, T, H, a.dx_add_stride, 2, false);
    ts.add("dx", a.dx, T, H, a.dx_stride, 2, true);
    ts.add("dw", a.dw, E, H, H, 4, true);
    ts.add("workspace", a.workspace, 1, need, need, 1, true);
    if ((rc = ts.check("dx", "dx_add")) || (rc = check_device(T > 0 ? (const void*)a.dlogits : a.dw, stream))) return rc;
    launch_router_logits_backward(a, (hipStream_t)stream);
    return launched();
}

int mega_moe_router_topk(const mega_moe_router_topk_args* args, void* stream) {
    if (!args) return bad("the argument block is NULL");
    mega_moe_router_topk_args a = *args;
    int rc = check_router(a);
    if (rc) return rc;
    if (a.num_topk > a.num_experts) return bad("num_topk is larger than num_experts");
    if (a.renormalize != 0 && a.renormalize != 1) return bad("renormalize must be 0 or 1");
    if (!std::isfinite(a.weight_scale)) return bad("weight_scale must be finite");
    if (a.num_groups < 0 || a.num_groups > ROUTER_MAX_GROUPS || (a.num_groups > 1 && a.num_experts % a.num_groups))
        return fail(MEGA_MOE_ERR_INVALID_ARG, "num_groups must divide num_experts and be at most %d, got %d",
                    ROUTER_MAX_GROUPS, a.num_groups);
    if (a.num_groups > 1) {
        const int size = a.num_experts / a.num_groups;
        if (a.topk_groups < 1 || a.topk_groups > a.num_groups) return bad("topk_groups must be in [1, num_groups]");
        if (a.topk_groups * size < a.num_topk) return bad("topk_groups hold fewer than num_topk experts");
        if (a.group_top < 1 || a.group_top > 2 || a.group_top > size)
            return bad("group_top must be 1 or 2, and at most the experts of a group");
    }
    if (a.weight_scale == 0.0f) a.weight_scale = 1.0f;
    if (a.num_tokens == 0) return ok();
    if (!a.logits || !a.topk_idx || !a.topk_weights) return bad("logits, topk_idx or topk_weights is NULL");
    if (!aligned(a.logits, type_bytes(a.logits_type)) || !words_aligned({a.bias, a.topk_idx, a.topk_weights}))
        return bad("logits must be aligned to their type, bias, topk_idx and topk_weights 4-byte");
    const int64_t T = a.num_tokens, E = a.num_experts, k = a.num_topk;
    a.logits_stride = stride_of(a.logits_stride, E, 1);
    if (a.logits_stride < 0) return bad("logits_stride is shorter than its row");
    Tensors ts;
    ts.add("logits", a.logits, T, E, a.logits_stride, type_bytes(a.logits_type), false);
    ts.add("bias", a.bias, 1, E, E, 4, false);
    ts.add("token_mask", a.token_mask, 1, T, T, 1, false);
    ts.add("topk_idx", a.topk_idx, T, k, k, 4, true);
    ts.add("topk_weights", a.topk_weights, T, k, k, 4, true);
    if ((rc = ts.check()) || (rc = check_device(a.logits, stream))) return rc;
    launch_router_topk(a, (hipStream_t)stream);
    return launched();
}

int64_t mega_moe_balance_loss_workspace_bytes(const mega_moe_balance_loss_args* a) {
    if (check_balance_sizes(a)) return -1;
    return balance_loss_workspace(*a);
}

int mega_moe_balance_loss(const mega_moe_balance_loss_args* args, void* stream) {
    int rc = check_balance_sizes(args);
    if (rc) return rc;
    mega_moe_balance_loss_args a = *args;
    if (!a.loss || !a.counts || !a.tokens) return bad("loss, counts or tokens is NULL");
    if (a.num_tokens > 0 && (!a.logits || !a.topk_idx)) return bad("logits or topk_idx is NULL");
    if (!aligned(a.logits, type_bytes(a.logits_type)) ||
        !words_aligned({a.topk_idx, a.cu_seqlens, a.loss, a.counts, a.tokens, a.probs}))
        return bad("logits must be aligned to their type, the other arrays 4-byte");
    const int64_t T = a.num_tokens, E = a.num_experts, k = a.num_topk, B = a.cu_seqlens ? a.num_sequences : 1;
    a.logits_stride = stride_of(a.logits_stride, E, 1);
    if (a.logits_stride < 0) return bad("logits_stride is shorter than its row");
    const int64_t need = balance_loss_workspace(a);
    if ((rc = check_workspace(a.workspace, a.workspace_bytes, need))) return rc;
    Tensors ts;
    ts.add("logits", a.logits, T, E, a.logits_stride, type_bytes(a.logits_type), false);
    ts.add("topk_idx", a.topk_idx, T, k, k, 4, false);
    ts.add("token_mask", a.token_mask, 1, T, T, 1, false);
    ts.add("cu_seqlens", a.cu_seqlens, 1, B + 1, B + 1, 4, false);
    ts.add("loss", a.loss, 1, 2, 2, 4, true);
    ts.add("counts", a.counts, B, E, E, 4, true);
    ts.add("tokens", a.tokens, 1, B + 2, B + 2, 4, true);
    ts.add("probs", a.probs, B, E, E, 4, true);
    ts.add("workspace", a.workspace, 1, need, need, 1, true);
    if ((rc = ts.check()) || (rc = check_device(a.loss, stream))) return rc;
    launch_balance_loss(a, (hipStream_t)stream);
    return launched();
}

int mega_moe_router_backward(const mega_moe_router_backward_args* args, void* stream) {
    if (!args) return bad("the argument block is NULL");
    mega_moe_router_backward_args a = *args;
    int rc = check_router(a);
    if (rc) return rc;
    if (a.renormalize != 0 && a.renormalize != 1) return bad("renormalize must be 0 or 1");
    if (!std::isfinite(a.weight_scale)) return bad("weight_scale must be finite");
    if (a.weight_scale == 0.0f) a.weight_scale = 1.0f;
    if ((rc = check_sequences(a))) return rc;
    if (!a.dweights && !a.dloss) return bad("dweights and dloss are both NULL");
    if (a.num_tokens == 0) return ok();
    if (!a.logits || !a.dlogits) return bad("logits or dlogits is NULL");
    if (a.dweights && !a.topk_idx) return bad("dweights needs topk_idx");
    if (a.dloss && (!a.counts || !a.tokens)) return bad("dloss needs counts and tokens");
    if (!aligned(a.logits, type_bytes(a.logits_type)) ||
        !words_aligned({a.topk_idx, a.dweights, a.dloss, a.cu_seqlens, a.counts, a.tokens, a.dlogits}))
        return bad("logits must be aligned to their type, the other arrays 4-byte");
    const int64_t T = a.num_tokens, E = a.num_experts, k = a.num_topk, B = a.cu_seqlens ? a.num_sequences : 1;
    a.logits_stride = stride_of(a.logits_stride, E, 1);
    a.dlogits_stride = stride_of(a.dlogits_stride, E, 1);
    if (a.logits_stride < 0 || a.dlogits_stride < 0) return bad("a stride is shorter than its row");
    Tensors ts;
    ts.add("logits", a.logits, T, E, a.logits_stride, type_bytes(a.logits_type), false);
    ts.add("topk_idx", a.topk_idx, T, k, k, 4, false);
    ts.add("token_mask", a.token_mask, 1, T, T, 1, false);
    ts.add("dweights", a.dweights, T, k, k, 4, false);
    ts.add("dloss", a.dloss, 1, 2, 2, 4, false);
    ts.add("cu_seqlens", a.cu_seqlens, 1, B + 1, B + 1, 4, false);
    ts.add("counts", a.counts, B, E, E, 4, false);
    ts.add("tokens", a.tokens, 1, B + 2, B + 2, 4, false);
    ts.add("dlogits", a.dlogits, T, E, a.dlogits_stride, 4, true);
    if ((rc = ts.check()) || (rc = check_device(a.logits, stream))) return rc;
    launch_router_backward(a, (hipStream_t)stream);
    return launched();
}

}  // extern "C"
