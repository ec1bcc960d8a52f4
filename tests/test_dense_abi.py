"""Checks of the dense path next to the layer that need no GPU: the argument
blocks' layout, every refusal (all come before any HIP call; the pointers are
stand-ins that are never used), workspaces and the rotary frequencies."""

import math

import numpy as np
import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from oracle import dense
from tests import test_block_abi as block_abi

M = 1 << 26          # stand-in addresses, 64 MB apart


def test_argument_blocks_have_the_header_s_layout(monkeypatch):
    monkeypatch.setattr(block_abi, "BLOCKS", [
        B.mega_moe_product_args, B.mega_moe_quantize_args, B.mega_moe_swiglu_backward_args, B.mega_moe_rotary_args,
        B.mega_moe_rotary_backward_args, B.mega_moe_rotary_frequencies_args])
    block_abi.test_argument_blocks_have_the_header_s_layout()


def _product(**kw):
    f = dict(m=4, n=256, k=512, a=M, a_sf=2 * M, b=3 * M, b_sf=4 * M, add=5 * M, out=6 * M, workspace=7 * M, workspace_bytes=1 << 22)
    f.update(kw)
    return B.make_args(B.mega_moe_product_args, **f)


def _quantize(**kw):
    f = dict(num_tokens=5, columns=256, activation=1, scale=1, x=M, up=2 * M, h=3 * M, q=4 * M, q_sf=5 * M, qt=6 * M, qt_sf=7 * M)
    f.update(kw)
    return B.make_args(B.mega_moe_quantize_args, **f)


def _swiglu_backward(**kw):
    f = dict(num_tokens=5, columns=256, x=M, up=2 * M, dh=3 * M, dx=4 * M, dup=5 * M, q=6 * M, q_sf=7 * M, qt=8 * M, qt_sf=9 * M)
    f.update(kw)
    return B.make_args(B.mega_moe_swiglu_backward_args, **f)


def _rotary(**kw):
    f = dict(num_tokens=5, q_heads=4, k_heads=2, head_dim=64, rotary_dim=32, weight_type=1, q=M, k=2 * M, q_weight=3 * M,
             k_weight=4 * M, positions=5 * M, inv_freq=6 * M, q_out=7 * M, k_out=8 * M)
    f.update(kw)
    return B.make_args(B.mega_moe_rotary_args, **f)


def _rotary_backward(**kw):
    f = dict(num_tokens=5, q_heads=4, k_heads=2, head_dim=64, rotary_dim=32, weight_type=1, q=M, k=2 * M, q_weight=3 * M,
             k_weight=4 * M, positions=5 * M, inv_freq=6 * M, dq_out=7 * M, dk_out=8 * M, dq=9 * M, dk=10 * M,
             dq_weight=11 * M, dk_weight=12 * M, workspace=13 * M, workspace_bytes=1 << 22)
    f.update(kw)
    return B.make_args(B.mega_moe_rotary_backward_args, **f)


HEADS = [dict(q_heads=-1), dict(q_heads=1025), dict(q_heads=0, k_heads=0, q_weight=None, k_weight=None), dict(k_heads=-2),
         dict(head_dim=0), dict(head_dim=60), dict(rotary_dim=8), dict(rotary_dim=80), dict(rotary_dim=-16), dict(rotary_start=-8),
         dict(rotary_start=4), dict(rotary_start=40), dict(layout=2), dict(type=2), dict(weight_type=-1),
         dict(first_position=-1), dict(first_position=2 ** 31 - 1), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
         dict(scale=float("inf")), dict(scale=float("nan")), dict(q_heads=0), dict(k_heads=0), dict(q=None), dict(k=None),
         dict(inv_freq=None), dict(q=M + 8), dict(k=2 * M + 2), dict(q_weight=3 * M + 4), dict(positions=5 * M + 2),
         dict(inv_freq=6 * M + 1), dict(q_stride=248), dict(q_stride=260), dict(k_stride=-128), dict(q_head_stride=56),
         dict(q_head_stride=68), dict(q_head_stride=(1 << 20) + 8), dict(q_head_stride=128, q_stride=256), dict(q_stride=2 ** 38 + 8)]
TOKENS = [dict(num_tokens=-1), dict(num_tokens=(1 << 21) + 1)]
COLUMNS = [dict(columns=0), dict(columns=64), dict(columns=200), dict(columns=(1 << 17) + 128), dict(x_type=2),
           dict(activation_clamp=-1.0), dict(activation_clamp=float("nan")), dict(q_sf=None), dict(qt=None)]
REFUSED = {
    "mega_moe_product": (_product, [
        dict(m=-1), dict(m=(1 << 21) + 1), dict(n=-8), dict(n=12), dict(n=(1 << 21) + 8), dict(k=-128), dict(k=100),
        dict(k=(1 << 21) + 128), dict(b_scale=2), dict(out_type=2), dict(reserved=1), dict(a=None), dict(a_sf=None), dict(b=None),
        dict(b_sf=None), dict(out=None), dict(a=M + 8), dict(b=3 * M + 4), dict(a_sf=2 * M + 2), dict(b_sf=4 * M + 1),
        dict(add=5 * M + 8), dict(out=6 * M + 2), dict(a_stride=256), dict(a_stride=520), dict(b_stride=-512), dict(a_sf_stride=3),
        dict(b_sf_stride=-4), dict(out_stride=128), dict(add_stride=260), dict(out=5 * M, out_stride=264), dict(out=M),
        dict(out=3 * M + 64), dict(add=6 * M + 16), dict(out=2 * M), dict(out=4 * M)]),
    "mega_moe_quantize": (_quantize, TOKENS + COLUMNS + [
        dict(activation=2), dict(scale=2), dict(activation=0), dict(activation=0, up=None, activation_clamp=1.0),
        dict(h=None, q=None, q_sf=None, qt=None, qt_sf=None), dict(x=None), dict(up=None), dict(x=M + 4), dict(up=2 * M + 8),
        dict(h=3 * M + 2), dict(q=4 * M + 8), dict(qt=6 * M + 4), dict(q_sf=5 * M + 2), dict(qt_sf=7 * M + 1), dict(x_stride=128),
        dict(up_stride=260), dict(h_stride=-256), dict(h=M), dict(q=2 * M), dict(qt=4 * M + 256), dict(qt_sf=5 * M), dict(h=M + 512)]),
    "mega_moe_swiglu_backward": (_swiglu_backward, TOKENS + COLUMNS + [
        dict(dx=None, dup=None, q=None, q_sf=None, qt=None, qt_sf=None), dict(x=None), dict(up=None), dict(dh=None), dict(x=M + 4),
        dict(dh=3 * M + 8), dict(dx=4 * M + 2), dict(dup=5 * M + 8), dict(q=6 * M + 8), dict(qt=8 * M + 4), dict(q_sf=7 * M + 2),
        dict(dh_stride=128), dict(dx_stride=260), dict(dup_stride=-256), dict(dx=M), dict(dup=4 * M + 256), dict(dx=3 * M),
        dict(q=8 * M), dict(qt_sf=7 * M + 16)]),
    "mega_moe_rotary": (_rotary, TOKENS + HEADS + [
        dict(q_out=None), dict(k_out=None), dict(q_out=7 * M + 2), dict(k_out_head_stride=56), dict(q_out=M, q_out_stride=512),
        dict(k_out=2 * M, k_out_head_stride=128), dict(q_out=2 * M), dict(k_out=M), dict(k_out=7 * M + 512), dict(q_out=M + 16)]),
    "mega_moe_rotary_backward": (_rotary_backward, TOKENS + HEADS + [
        dict(q_weight=None), dict(k_weight=None), dict(dq_out=None), dict(dk_out=None), dict(dq=None), dict(dk=None),
        dict(dq_out=7 * M + 8), dict(dk=10 * M + 4), dict(dq_weight=11 * M + 2), dict(dq_head_stride=8), dict(dk_out_stride=64),
        dict(dq=7 * M, dq_stride=512), dict(dk=8 * M, dk_head_stride=128), dict(dq=M), dict(dk=9 * M), dict(dq_weight=12 * M),
        dict(workspace=None), dict(workspace_bytes=8), dict(workspace=13 * M + 4), dict(workspace=9 * M)]),
}


@pytest.mark.parametrize("name,change", [(n, c) for n, (_, cs) in REFUSED.items() for c in cs],
                         ids=lambda v: v if isinstance(v, str) else "-".join(f"{k}={x}" for k, x in v.items()))
def test_call_is_refused(name, change):
    with pytest.raises(B.MegaMoEError) as ei:
        getattr(B, name)(REFUSED[name][0](**change), None)
    assert ei.value.code == B.MEGA_MOE_ERR_INVALID_ARG
    assert B.mega_moe_last_error()


@pytest.mark.parametrize("name,change", [
    ("mega_moe_product", dict(a_stride=(1 << 22) + 16, m=1)), ("mega_moe_product", dict(b_stride=(1 << 22) + 16)),
    ("mega_moe_product", dict(a_sf_stride=(1 << 20) + 1)), ("mega_moe_product", dict(b_sf_stride=(1 << 20) + 1)),
    ("mega_moe_rotary", dict(head_dim=520)), ("mega_moe_rotary_backward", dict(head_dim=1024))])
def test_what_is_not_built_is_unsupported(name, change):
    with pytest.raises(B.MegaMoEError) as ei:
        getattr(B, name)(REFUSED[name][0](**change), None)
    assert ei.value.code == B.MEGA_MOE_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", list(REFUSED))
def test_call_without_a_block_is_refused_and_without_rows_is_none(name):
    with pytest.raises(B.MegaMoEError) as ei:
        getattr(B, name)(None, None)
    assert ei.value.code == B.MEGA_MOE_ERR_INVALID_ARG
    none = dict(m=0) if name == "mega_moe_product" else dict(num_tokens=0)
    if name == "mega_moe_rotary_backward":
        none.update(dq_weight=None, dk_weight=None)
    assert getattr(B, name)(REFUSED[name][0](**none), None) == 0


def test_good_calls_pass_the_checks_and_stop_at_the_device():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: stand-in pointers must not reach it")
    packed = dict(q=M, k=M + 512, q_stride=512, k_stride=512, q_out=M, k_out=M + 512, q_out_stride=512, k_out_stride=512)
    for call, args in ((B.mega_moe_product, _product()), (B.mega_moe_product, _product(add=6 * M)), (B.mega_moe_product, _product(add=None)),
                       (B.mega_moe_product, _product(k=0, a=None, a_sf=None, b=None, b_sf=None)), (B.mega_moe_quantize, _quantize()),
                       (B.mega_moe_quantize, _quantize(up=M + 512, x_stride=512, up_stride=512)),
                       (B.mega_moe_quantize, _quantize(activation=0, up=None, scale=0)), (B.mega_moe_swiglu_backward, _swiglu_backward()),
                       (B.mega_moe_swiglu_backward, _swiglu_backward(dup=4 * M + 512, dx_stride=512, dup_stride=512)),
                       (B.mega_moe_rotary, _rotary()), (B.mega_moe_rotary, _rotary(**packed)),
                       (B.mega_moe_rotary, _rotary(k_heads=0, k=None, k_weight=None, k_out=None)), (B.mega_moe_rotary_backward, _rotary_backward()),
                       (B.mega_moe_rotary_backward, _rotary_backward(dq=7 * M, dk=8 * M)),
                       (B.mega_moe_rotary_backward, _rotary_backward(q=None, q_weight=None, dq_weight=None))):
        with pytest.raises(B.MegaMoEError) as ei:
            call(args, None)
        assert ei.value.code in (B.MEGA_MOE_ERR_HIP, B.MEGA_MOE_ERR_UNSUPPORTED), B.mega_moe_last_error()


# heads of q, k and v in turn: [tokens, heads, 3, 64]
IN_TURN = dict(q_heads=4, k_heads=4, q=M, k=M + 128)
IN_TURN_STRIDES = dict(q_stride=768, k_stride=768, q_head_stride=192, k_head_stride=192)


@pytest.mark.parametrize("kw,good", [
    (dict(q_out=M, k_out=M + 128), True), (dict(q_out=7 * M, k_out=7 * M + 128), True), (dict(q_out=M + 256, k_out=7 * M), True),
    (dict(q_out=M + 64, k_out=7 * M), False), (dict(q_out=7 * M, k_out=7 * M + 112), False), (dict(q_out=M + 128, k_out=M), False),
    (dict(q_out=7 * M, k_out=7 * M + 128, q_out_stride=776), False), (dict(q_out=M, k_out=M + 128, k_out_head_stride=128), False)])
def test_heads_in_turn_pass_the_checks_where_they_do_not_meet(kw, good):
    if good and torch.cuda.is_available():
        pytest.skip("a GPU is present: stand-in pointers must not reach it")
    args = _rotary(**IN_TURN, **IN_TURN_STRIDES, **{**dict(q_out_stride=768, k_out_stride=768, q_out_head_stride=192, k_out_head_stride=192), **kw})
    with pytest.raises(B.MegaMoEError) as ei:
        B.mega_moe_rotary(args, None)
    assert (ei.value.code == B.MEGA_MOE_ERR_INVALID_ARG) == (not good), B.mega_moe_last_error()


def test_workspace_bytes_need_no_gpu_and_refuse_bad_sizes():
    assert B.mega_moe_product_workspace_bytes(_product(a=None, workspace=None)) >= 0
    assert B.mega_moe_product_workspace_bytes(_product(k=0)) == 0
    assert B.mega_moe_product_workspace_bytes(_product(n=4)) == -1
    assert B.mega_moe_product_workspace_bytes(_product(k=1 << 21, m=1 << 21, n=1 << 21)) >= 0
    assert B.mega_moe_rotary_workspace_bytes(_rotary_backward(workspace=None)) > 0
    assert B.mega_moe_rotary_workspace_bytes(_rotary_backward(dq_weight=None, dk_weight=None)) == 0
    assert B.mega_moe_rotary_workspace_bytes(_rotary_backward(head_dim=4)) == -1


def _frequencies(dim=64, **kw):
    inv, scale = torch.full((max(dim, 2) // 2 + 1,), 7.0), torch.zeros(1)
    f = dict(rotary_dim=dim, base=10000.0, inv_freq=inv, scale=scale)
    f.update(kw)
    B.mega_moe_rotary_frequencies(B.make_args(B.mega_moe_rotary_frequencies_args, **f))
    assert inv[-1] == 7.0
    return inv[:-1].numpy(), float(scale)


@pytest.mark.parametrize("dim", [16, 64, 128, 512])
@pytest.mark.parametrize("base", [500.0, 10000.0, 8e6])
def test_frequencies_are_those_of_the_formulas(dim, base):
    half = 2.0 ** -24
    for kw, want in (
            (dict(), dense.frequencies(dim, base)),
            (dict(scaling=B.MEGA_MOE_ROTARY_LINEAR, factor=8.0), dense.frequencies(dim, base, factor=8.0)),
            (dict(scaling=B.MEGA_MOE_ROTARY_BY_PARTS, factor=40.0, original_length=4096.0, fast_turns=32.0, slow_turns=1.0),
             dense.frequencies(dim, base, 40.0, 4096.0, 32.0, 1.0))):
        inv, scale = _frequencies(dim, base=base, **kw)
        np.testing.assert_allclose(inv, want[0], rtol=half + 1e-12, atol=0)
        assert abs(scale - want[1]) <= half * want[1]


def test_frequencies_by_parts_keep_the_fast_and_divide_the_slow():
    inv, scale = _frequencies(128, scaling=B.MEGA_MOE_ROTARY_BY_PARTS, factor=8.0, original_length=4096.0, fast_turns=32.0, slow_turns=1.0)
    plain, _ = _frequencies(128)
    turns = 4096.0 * plain / (2 * math.pi)
    assert (turns > 32).any() and (turns < 1).any()
    fast, slow = turns > 32 * 1.2, turns < 1 / 1.2
    assert (inv[fast] == plain[fast]).all()
    np.testing.assert_allclose(inv[slow], plain[slow] / 8, rtol=2.0 ** -23)
    assert ((inv <= plain) & (inv >= plain / 8 * (1 - 2.0 ** -23))).all()
    assert scale == pytest.approx(0.1 * math.log(8.0) + 1.0, rel=2.0 ** -24)


@pytest.mark.parametrize("kw", [
    dict(dim=8), dict(dim=0), dict(dim=528), dict(scaling=3), dict(scaling=-1), dict(base=1.0), dict(base=float("inf")), dict(base=0.0),
    dict(factor=2.0), dict(scaling=1), dict(scaling=1, factor=0.5), dict(scaling=1, factor=float("nan")),
    dict(scaling=2, factor=2.0), dict(scaling=2, factor=2.0, original_length=100.0, fast_turns=1.0, slow_turns=1.0),
    dict(scaling=2, factor=2.0, original_length=100.0, fast_turns=1.0), dict(scaling=2, factor=2.0, original_length=float("inf"),
                                                                             fast_turns=2.0, slow_turns=1.0), dict(inv_freq=None)],
    ids=str)
def test_frequencies_are_refused(kw):
    with pytest.raises(B.MegaMoEError) as ei:
        _frequencies(**kw)
    assert ei.value.code == B.MEGA_MOE_ERR_INVALID_ARG


def test_frequencies_without_a_block_are_refused():
    with pytest.raises(B.MegaMoEError):
        B.mega_moe_rotary_frequencies(None)
