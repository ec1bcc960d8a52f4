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


@pytest.mark.parametrize("tokens", [4097, 4500, 8400])
def test_gradients_of_several_runs_of_tokens(tokens):
    # 512 rotated columns: a workgroup of 256 has 16 tokens' turns at a time, and goes on to further ones
    g = D.generator(tokens)
    dim, make = 512, lambda scale: D.randn(g, tokens, 2, dim, scale=scale, dtype=torch.bfloat16)   # noqa: E731
    x, d, dx = make(1.5), make(0.5), torch.zeros(tokens, 2, dim, dtype=torch.bfloat16, device="cuda")
    freq = torch.tensor([10000.0 ** (-2 * i / dim) for i in range(dim // 2)], device="cuda")
    weight, dw = 1 + D.randn(g, 2, dim, scale=0.1), torch.zeros(2, dim, device="cuda")
    strides = {f"{n}_stride": 2 * dim for n in ("q", "k", "dq_out", "dk_out", "dq", "dk")}
    args = B.make_args(B.mega_moe_rotary_backward_args, num_tokens=tokens, q_heads=1, k_heads=1, head_dim=dim, rotary_dim=dim,
                       weight_type=B.MEGA_MOE_F32, eps=1e-6, inv_freq=freq, q=x[:, 0], k=x[:, 1], q_weight=weight[0], k_weight=weight[1],
                       dq_out=d[:, 0], dk_out=d[:, 1], dq=dx[:, 0], dk=dx[:, 1], dq_weight=dw[0], dk_weight=dw[1], **strides)
    B.set_args(args, **U.workspace(B.mega_moe_rotary_workspace_bytes(args)))
    B.mega_moe_rotary_backward(args, U.current_stream())
    for i in range(2):
        want = dense.rotary_backward(U.f64(x[:, i:i + 1]), U.f64(weight[i]), U.f64(d[:, i:i + 1]), range(tokens), U.f64(freq), eps=1e-6)
        U.near(dx[:, i:i + 1], want[0], want[1], 64, f"gradients {i}")
        # a thread's run of items, 16 groups, a column of 16 rows and 64 of their sums
        U.near(dw[i], want[2], want[3], 64 + tokens // 16 + 128, f"weight {i}")
