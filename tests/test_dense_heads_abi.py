"""Calls of the heads' operators that the checks must let through: what belongs
to heads that a call does not have is not looked at, and positions go up to the
largest 32-bit number.  No GPU: the pointers are stand-ins."""

import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from tests.test_dense_abi import M, _rotary, _rotary_backward

CALLS = {"rotary": (B.mega_moe_rotary, _rotary), "rotary_backward": (B.mega_moe_rotary_backward, _rotary_backward)}
NO_Q = dict(q_heads=0, q=None, q_weight=None)
NO_K = dict(k_heads=0, k=None, k_weight=None)
OUT = {"rotary": {"q": dict(q_out=None), "k": dict(k_out=None)},
       "rotary_backward": {"q": dict(dq_out=None, dq=None, dq_weight=None), "k": dict(dk_out=None, dk=None, dk_weight=None)}}
# left over from a packed projection, and of no use at all
LEFT = [dict(k_stride=512, k_out_stride=256), dict(k_stride=8), dict(k_head_stride=12), dict(k_stride=-1, k_head_stride=-8),
        dict(k_head_stride=64, k_out_head_stride=128)]


def _code(call, args):
    """The refusal's code; a call that the checks let through stops at the device."""
    with pytest.raises(B.MegaMoEError) as ei:
        call(args, None)
    return ei.value.code


def _no_gpu():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: stand-in pointers must not reach it")


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("side", ["q", "k"])
@pytest.mark.parametrize("left", LEFT, ids=str)
def test_strides_of_heads_that_are_not_there_are_not_looked_at(name, side, left):
    _no_gpu()
    call, make = CALLS[name]
    f = {**(NO_K if side == "k" else NO_Q), **OUT[name][side]}
    for key, v in left.items():
        key = side + key[1:]
        f["d" + key if name == "rotary_backward" and "_out" in key else key] = v
    assert _code(call, make(**f)) in (B.MEGA_MOE_ERR_HIP, B.MEGA_MOE_ERR_UNSUPPORTED), B.mega_moe_last_error()


@pytest.mark.parametrize("name", list(CALLS))
def test_strides_of_heads_in_place_still_have_to_agree(name):
    call, make = CALLS[name]
    f = dict(q_out=M, q_out_stride=512) if name == "rotary" else dict(dq=7 * M, dq_stride=512)
    assert _code(call, make(**f)) == B.MEGA_MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("tokens,first,good", [(1, 2 ** 31 - 1, True), (2, 2 ** 31 - 2, True), (5, 2 ** 31 - 5, True),
                                               (2, 2 ** 31 - 1, False), (5, 2 ** 31 - 4, False)])
def test_last_position_is_the_largest_32_bit_number(name, tokens, first, good):
    if good:
        _no_gpu()
    call, make = CALLS[name]
    code = _code(call, make(num_tokens=tokens, first_position=first, positions=None))
    assert (code == B.MEGA_MOE_ERR_INVALID_ARG) == (not good), B.mega_moe_last_error()
