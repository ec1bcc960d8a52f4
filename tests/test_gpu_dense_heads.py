"""The heads' operators at positions and strides that no other test has."""

import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from oracle import dense
from tests import block_util as U
from tests import dense_util as D

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 3])
def test_positions_up_to_the_largest_32_bit_number(tokens):
    g = D.generator(tokens)
    first, heads, dim = 2 ** 31 - tokens, 3, 64
    q, out, dq = D.randn(g, tokens, heads, dim), *(torch.zeros(tokens, heads, dim, device="cuda") for _ in range(2))
    freq = torch.tensor([10000.0 ** (-i / 32) for i in range(32)], device="cuda")
    weight, dw = 1 + D.randn(g, dim, scale=0.1), torch.zeros(dim, device="cuda")
    f = dict(num_tokens=tokens, q_heads=heads, head_dim=dim, rotary_dim=dim, type=B.MEGA_MOE_F32, weight_type=B.MEGA_MOE_F32, eps=1e-6,
             first_position=first, inv_freq=freq, q=q, q_weight=weight)
    # (no heads of k: their strides are of no matter)
    B.mega_moe_rotary(B.make_args(B.mega_moe_rotary_args, q_out=out, k_stride=512, k_out_stride=256, **f), U.current_stream())
    positions = [first + t for t in range(tokens)]
    want, mag = dense.rotary(U.f64(q), U.f64(weight), positions, U.f64(freq), eps=1e-6)
    U.near(out, want, mag, 40, "heads")
    d = D.randn(g, tokens, heads, dim)
    args = B.make_args(B.mega_moe_rotary_backward_args, dq_out=d, dq=dq, dq_weight=dw, k_stride=8, dk_stride=12, **f)
    B.set_args(args, **U.workspace(B.mega_moe_rotary_workspace_bytes(args)))
    B.mega_moe_rotary_backward(args, U.current_stream())
    want = dense.rotary_backward(U.f64(q), U.f64(weight), U.f64(d), positions, U.f64(freq), eps=1e-6)
    U.near(dq, want[0], want[1], 64, "dq")
    U.near(dw, want[2], want[3], 64 + 2 * tokens * heads, "dw")
