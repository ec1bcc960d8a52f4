"""Checks of the operators around the layer that need no GPU: the argument
blocks' layout, and every refusal (all of them come before any HIP call; the
pointers below are stand-ins that are never used)."""

import os
import subprocess
import tempfile

import pytest

from fp8_mixture_experts_amd import binding as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BLOCKS = [B.mega_moe_norm_args, B.mega_moe_norm_backward_args, B.mega_moe_router_logits_args,
          B.mega_moe_router_topk_args, B.mega_moe_balance_loss_args, B.mega_moe_router_backward_args]


def test_argument_blocks_have_the_header_s_layout():
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "mega_moe.h"', "int main(void) {"]
    for cls in BLOCKS:
        n = cls.__name__
        lines.append(f'printf("{n} %zu\\n", sizeof({n}));')
        lines += [f'printf("{n}.{f[0]} %zu %zu\\n", offsetof({n}, {f[0]}), sizeof((({n}*)0)->{f[0]}));' for f in cls._fields_]
    lines.append("return 0; }")
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "a.c"), os.path.join(d, "a")
        open(src, "w").write("\n".join(lines))
        subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), src, "-o", exe], check=True)
        got = subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split("\n")
    want = []
    import ctypes
    for cls in BLOCKS:
        want.append(f"{cls.__name__} {ctypes.sizeof(cls)}")
        want += [f"{cls.__name__}.{f[0]} {getattr(cls, f[0]).offset} {getattr(cls, f[0]).size}" for f in cls._fields_]
    assert got[:-1] == want


def test_argument_blocks_keep_tensors_and_know_their_fields():
    import torch
    t = torch.zeros(8)
    a = B.make_args(B.mega_moe_norm_args, h=t, hidden=8)
    assert a.h == t.data_ptr() and a.tensors["h"] is t
    B.set_args(a, h=None)
    assert a.h is None and "h" not in a.tensors
    with pytest.raises(AttributeError):
        B.set_args(a, nothing=1)


M = 1 << 20          # stand-in addresses, a megabyte apart


def _norm(**kw):
    f = dict(num_tokens=4, hidden=256, weight_type=1, gate_type=1, residual_scale=1.0, h=M, y=2 * M, post_weight=3 * M,
             pre_weight=4 * M, r=5 * M, n=6 * M, q=7 * M, q_sf=8 * M)
    f.update(kw)
    return B.make_args(B.mega_moe_norm_args, **f)


def _norm_backward(**kw):
    f = dict(num_tokens=4, hidden=256, weight_type=1, gate_type=1, residual_scale=1.0, r=M, y=2 * M, post_weight=3 * M,
             pre_weight=4 * M, dr=5 * M, dn=6 * M, dh=7 * M, dy=8 * M, dpost_weight=9 * M, dpre_weight=10 * M,
             workspace=11 * M, workspace_bytes=1 << 19)
    f.update(kw)
    return B.make_args(B.mega_moe_norm_backward_args, **f)


def _logits(**kw):
    f = dict(num_tokens=4, hidden=256, num_experts=8, x=M, w=2 * M, logits=3 * M, dlogits=4 * M, dx=5 * M, dw=6 * M,
             workspace=7 * M, workspace_bytes=1 << 19)
    f.update(kw)
    return B.make_args(B.mega_moe_router_logits_args, **f)


def _topk(**kw):
    f = dict(num_tokens=4, num_experts=8, num_topk=2, logits_type=1, logits=M, bias=2 * M, topk_idx=3 * M, topk_weights=4 * M)
    f.update(kw)
    return B.make_args(B.mega_moe_router_topk_args, **f)


def _balance(**kw):
    f = dict(num_tokens=4, num_experts=8, num_topk=2, logits_type=1, logits=M, topk_idx=2 * M, loss=3 * M, counts=4 * M,
             tokens=5 * M, probs=6 * M, workspace=7 * M, workspace_bytes=1 << 19)
    f.update(kw)
    return B.make_args(B.mega_moe_balance_loss_args, **f)


def _router_backward(**kw):
    f = dict(num_tokens=4, num_experts=8, num_topk=2, logits_type=1, logits=M, topk_idx=2 * M, dweights=3 * M, dloss=4 * M,
             counts=5 * M, tokens=6 * M, dlogits=7 * M)
    f.update(kw)
    return B.make_args(B.mega_moe_router_backward_args, **f)


SIZES = [dict(num_tokens=-1), dict(num_tokens=(1 << 21) + 1)]
REFUSED = {
    "mega_moe_norm": (_norm, SIZES + [
        dict(hidden=0), dict(hidden=260), dict(hidden=264), dict(stream_type=2), dict(weight_type=-1),
        dict(gate_type=5), dict(gate_kind=4), dict(gate_kind=-1), dict(reserved=1), dict(post_eps=-1.0),
        dict(pre_eps=float("nan")), dict(pre_eps=float("inf")), dict(residual_scale=float("inf")),
        dict(gate=9 * M), dict(gate_kind=1), dict(y=None), dict(y=None, post_weight=None, residual_scale=0.5),
        dict(pre_weight=None), dict(q=None), dict(q_sf=None), dict(r=None, n=None, q=None, q_sf=None), dict(h=None),
        dict(h=M + 8), dict(y=2 * M + 4), dict(r=5 * M + 8), dict(n=6 * M + 2), dict(q=7 * M + 8), dict(q_sf=8 * M + 2),
        dict(pre_weight=4 * M + 4), dict(h_stride=128), dict(h_stride=260), dict(n_stride=-256),
        dict(gate_kind=1, gate=9 * M + 2), dict(gate_kind=2, gate=9 * M + 4),
        dict(n=5 * M), dict(r=2 * M), dict(n=M + 512), dict(r=M, r_stride=264), dict(q_sf=7 * M + 16),
        dict(r=M + 16, h_stride=512, r_stride=512)]),
    "mega_moe_norm_backward": (_norm_backward, SIZES + [
        dict(hidden=12), dict(y=None), dict(dy=8 * M, y=None, post_weight=None, dpost_weight=None), dict(pre_weight=None),
        dict(post_weight=None), dict(dgate=12 * M), dict(dr=None, dn=None), dict(r=None),
        dict(dh=None, dy=None, dpost_weight=None, dpre_weight=None), dict(workspace=None), dict(workspace=11 * M + 4),
        dict(workspace_bytes=16), dict(dh=M), dict(dh=5 * M, dh_stride=512), dict(dy=6 * M), dict(dpre_weight=9 * M + 16),
        dict(workspace=7 * M), dict(dr_stride=100), dict(dpre_weight=10 * M + 4),
        dict(gate_kind=1, gate=12 * M, dgate=13 * M + 2), dict(gate_kind=2, gate=12 * M, dgate=13 * M + 4)]),
    "mega_moe_router_logits": (_logits, SIZES + [
        dict(hidden=4), dict(num_experts=0), dict(num_experts=1025), dict(weight_type=3), dict(x=None),
        dict(w=None), dict(logits=None), dict(x=M + 2), dict(w=2 * M + 8), dict(logits=3 * M + 1), dict(x_stride=255),
        dict(x_stride=260), dict(logits_stride=7), dict(logits=M), dict(logits=2 * M + 64)]),
    "mega_moe_router_logits_backward": (_logits, SIZES + [
        dict(dx=None, dw=None), dict(dx=None, dx_add=8 * M), dict(dlogits=None), dict(w=None), dict(x=None),
        dict(dx=5 * M + 4), dict(dw=6 * M + 8), dict(dlogits=4 * M + 2), dict(dlogits_stride=3), dict(dx_stride=8),
        dict(dx_add_stride=260), dict(dx=M), dict(dw=2 * M), dict(dw=5 * M + 256), dict(dx_add=5 * M, dx_add_stride=512)]),
    "mega_moe_router_topk": (_topk, SIZES + [
        dict(num_experts=0), dict(num_experts=2000), dict(num_topk=0), dict(num_topk=9), dict(logits_type=2), dict(score=2),
        dict(renormalize=2), dict(weight_scale=float("nan")), dict(num_groups=3), dict(num_groups=-2),
        dict(num_experts=130, num_groups=65), dict(num_groups=4, topk_groups=0, group_top=1),
        dict(num_groups=4, topk_groups=5, group_top=1), dict(num_groups=8, topk_groups=1, group_top=1),
        dict(num_groups=4, topk_groups=2, group_top=3), dict(num_groups=8, topk_groups=4, group_top=2),
        dict(logits=None), dict(topk_idx=None), dict(topk_weights=None), dict(logits=M + 2), dict(bias=2 * M + 1),
        dict(topk_idx=3 * M + 2), dict(logits_stride=4), dict(topk_idx=M), dict(topk_weights=3 * M + 16)]),
    "mega_moe_balance_loss": (_balance, SIZES + [
        dict(num_experts=0), dict(num_topk=0), dict(num_topk=1025), dict(num_topk=2 ** 31 - 1), dict(score=-1),
        dict(logits_stride=2 ** 38 + 1), dict(num_sequences=2), dict(cu_seqlens=8 * M),
        dict(num_sequences=-1), dict(num_sequences=(1 << 21) + 1, cu_seqlens=8 * M), dict(balance_coeff=float("inf")),
        dict(z_coeff=float("nan")), dict(loss=None), dict(counts=None), dict(tokens=None), dict(logits=None),
        dict(topk_idx=None), dict(loss=3 * M + 2), dict(logits=M + 2), dict(workspace=None), dict(workspace_bytes=8),
        dict(workspace=7 * M + 8), dict(counts=2 * M), dict(probs=4 * M), dict(logits_stride=5)]),
    "mega_moe_router_backward": (_router_backward, SIZES + [
        dict(num_experts=1025), dict(num_topk=0), dict(num_topk=2 ** 31 - 1), dict(renormalize=-1), dict(weight_scale=float("inf")),
        dict(dweights=None, dloss=None), dict(logits=None), dict(dlogits=None), dict(topk_idx=None), dict(counts=None),
        dict(tokens=None), dict(num_sequences=3), dict(cu_seqlens=8 * M), dict(dlogits=M), dict(dlogits=3 * M),
        dict(dlogits_stride=4), dict(dlogits=7 * M + 2)]),
}


@pytest.mark.parametrize("name,change", [(n, c) for n, (_, cs) in REFUSED.items() for c in cs],
                         ids=lambda v: v if isinstance(v, str) else "-".join(f"{k}={x}" for k, x in v.items()))
def test_call_is_refused(name, change):
    make = REFUSED[name][0]
    with pytest.raises(B.MegaMoEError) as ei:
        getattr(B, name)(make(**change), None)
    assert ei.value.code == B.MEGA_MOE_ERR_INVALID_ARG
    assert B.mega_moe_last_error()


@pytest.mark.parametrize("name", [n for n in REFUSED if "norm" in n or "logits" in n])
def test_hidden_beyond_what_is_built_is_unsupported(name):
    with pytest.raises(B.MegaMoEError) as ei:
        getattr(B, name)(REFUSED[name][0](hidden=8320), None)
    assert ei.value.code == B.MEGA_MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["mega_moe_router_logits", "mega_moe_router_logits_backward"])
def test_rows_of_x_too_far_apart_are_unsupported(name):
    with pytest.raises(B.MegaMoEError) as ei:
        getattr(B, name)(_logits(x_stride=(1 << 22) + 8, num_tokens=1), None)
    assert ei.value.code == B.MEGA_MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", list(REFUSED))
def test_call_without_a_block_is_refused_and_without_tokens_is_none(name):
    with pytest.raises(B.MegaMoEError) as ei:
        getattr(B, name)(None, None)
    assert ei.value.code == B.MEGA_MOE_ERR_INVALID_ARG
    if name in ("mega_moe_norm", "mega_moe_router_logits", "mega_moe_router_topk", "mega_moe_router_backward"):
        assert getattr(B, name)(REFUSED[name][0](num_tokens=0), None) == 0


def test_good_calls_pass_the_checks_and_stop_at_the_device():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: stand-in pointers must not reach it")
    side = dict(r=M + 512, h_stride=512, r_stride=512)        # columns 256 .. 511 of one wider array
    for call, args in ((B.mega_moe_norm, _norm()), (B.mega_moe_norm, _norm(r=M)), (B.mega_moe_norm, _norm(**side)),
                       (B.mega_moe_norm_backward, _norm_backward()), (B.mega_moe_norm_backward, _norm_backward(dh=5 * M)),
                       (B.mega_moe_router_logits, _logits()), (B.mega_moe_router_logits_backward, _logits()),
                       (B.mega_moe_router_logits_backward, _logits(dx_add=5 * M)), (B.mega_moe_router_topk, _topk()),
                       (B.mega_moe_balance_loss, _balance()), (B.mega_moe_router_backward, _router_backward())):
        with pytest.raises(B.MegaMoEError) as ei:
            call(args, None)
        assert ei.value.code in (B.MEGA_MOE_ERR_HIP, B.MEGA_MOE_ERR_UNSUPPORTED), B.mega_moe_last_error()


def test_workspace_bytes_need_no_gpu_and_refuse_bad_sizes():
    assert B.mega_moe_norm_workspace_bytes(_norm_backward(workspace=None)) > 0
    assert B.mega_moe_norm_workspace_bytes(_norm_backward(dpost_weight=None, dpre_weight=None)) == 0
    assert B.mega_moe_norm_workspace_bytes(_norm_backward(hidden=4)) == -1
    assert B.mega_moe_router_logits_workspace_bytes(_logits()) >= 0
    assert B.mega_moe_router_logits_workspace_bytes(_logits(num_experts=0)) == -1
    assert B.mega_moe_balance_loss_workspace_bytes(_balance()) > 0
    assert B.mega_moe_balance_loss_workspace_bytes(_balance(num_topk=0)) == -1


@pytest.mark.parametrize("experts,most", [(32, 1 << 21), (224, 1 << 21), (225, (1 << 21) - 1), (256, (1 << 21) - 1), (1024, (1 << 19) - 1)])
def test_more_sequences_than_a_launch_has_workgroups_for_are_unsupported(experts, most):
    # the second launch has a workgroup of 256 threads for 32 experts of a sequence,
    # and a launch fewer than 2^32 threads
    G = 1 << 36          # stand-in addresses further apart than the arrays are long

    def call(n):
        return _balance(num_experts=experts, num_sequences=n, logits=G, topk_idx=2 * G, loss=3 * G, counts=4 * G, tokens=5 * G,
                        probs=6 * G, cu_seqlens=7 * G, workspace=8 * G, workspace_bytes=1 << 40)

    assert B.mega_moe_balance_loss_workspace_bytes(call(most)) > 0
    if most < 1 << 21:
        assert B.mega_moe_balance_loss_workspace_bytes(call(most + 1)) == -1
        with pytest.raises(B.MegaMoEError) as ei:
            B.mega_moe_balance_loss(call(most + 1), None)
        assert ei.value.code == B.MEGA_MOE_ERR_UNSUPPORTED and "num_sequences" in B.mega_moe_last_error()
