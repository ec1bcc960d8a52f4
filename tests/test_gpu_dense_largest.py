"""The dense path's operators at the largest counts that their arguments allow."""

import numpy as np
import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from oracle import dense
from tests import block_util as U
from tests import dense_util as D
from tests.test_gpu_dense import _check_quantize, _quantize, _swiglu_backward
from tests.test_gpu_dense_tiles import _reference

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
MOST = 2 ** 21


@pytest.mark.parametrize("m,k,n", [(MOST, 128, 8), (MOST - 5, 128, 24), (1, 128, MOST), (16, 256, MOST - 8), (3, MOST, 24), (40, MOST, 8)])
@pytest.mark.parametrize("out_type", [BF16, F32], ids=["bf16", "f32"])
def test_product_of_the_most_rows_and_columns(m, k, n, out_type):
    scale = "row" if k == MOST else "block"
    g = D.generator(m + n)
    a, a_sf = D.operand(g, m, k)
    b, b_sf = D.operand(g, n, k, scale)
    buf = torch.full((m + 1, n), 7.0, dtype=out_type, device="cuda")
    D.product(a, a_sf, b, b_sf, buf[:m], scale)
    D.check_product(buf[:m], a, a_sf, b, b_sf, scale, ref=_reference(a, a_sf, b, b_sf, scale))
    assert bool((buf[m] == 7).all())


@pytest.mark.parametrize("scale", ["row", "block"])
def test_codes_of_the_most_columns(scale):
    g = D.generator(1)
    x = D.randn(g, 130, 2 ** 17, dtype=BF16)
    _check_quantize(_quantize(x, None, scale), U.f64(x), scale, 0)
    if scale == "row":
        both = D.randn(g, 5, 2 ** 18, scale=2.0, dtype=BF16)
        gate, up, dh = both[:, :2 ** 17], both[:, 2 ** 17:], D.randn(g, 5, 2 ** 17, scale=1e-2, dtype=BF16)
        o = _swiglu_backward(gate, up, dh)
        dx, dx_mag, dup, dup_mag = dense.swiglu_backward(U.f64(gate), U.f64(up), U.f64(dh))
        U.near(o["dx"], dx, dx_mag, 16, "dx")
        U.near(o["dup"], dup, dup_mag, 16, "dup")
        v, mag = np.concatenate([dx, dup], axis=1), np.concatenate([dx_mag, dup_mag], axis=1)
        D.check_codes(o["q"], o["q_sf"], dense.rows_quotients(v, mag), 16, "q")
        D.check_codes(o["qt"], o["qt_sf"], dense.transposed_quotients(v, mag), 16, "qt")


@pytest.mark.parametrize("tokens,heads,dim", [(MOST, 1, 16), (5, 1024, 16)])
def test_heads_of_the_most_tokens_and_heads(tokens, heads, dim):
    g = D.generator(heads)
    q, k = (D.randn(g, tokens, heads, dim, dtype=BF16) for _ in range(2))
    freq = torch.tensor([10000.0 ** (-2 * i / dim) for i in range(dim // 2)], device="cuda")
    weight = 1 + D.randn(g, 2, dim, scale=0.1)
    f = dict(num_tokens=tokens, q_heads=heads, k_heads=heads, head_dim=dim, rotary_dim=dim, weight_type=B.MEGA_MOE_F32, eps=1e-6,
             inv_freq=freq, q_weight=weight[0], k_weight=weight[1], q=q, k=k)
    qo, ko, dq, dk = (torch.zeros_like(q) for _ in range(4))
    dw = torch.zeros(2, dim, device="cuda")
    B.mega_moe_rotary(B.make_args(B.mega_moe_rotary_args, q_out=qo, k_out=ko, **f), U.current_stream())
    d = [D.randn(g, tokens, heads, dim, dtype=BF16) for _ in range(2)]
    args = B.make_args(B.mega_moe_rotary_backward_args, dq_out=d[0], dk_out=d[1], dq=dq, dk=dk, dq_weight=dw[0], dk_weight=dw[1], **f)
    B.set_args(args, **U.workspace(B.mega_moe_rotary_workspace_bytes(args)))
    B.mega_moe_rotary_backward(args, U.current_stream())
    # the first and last tokens; the weights' sums over all of them in float64 on the GPU
    some = [t for t in (*range(40), *range(tokens // 2, tokens // 2 + 40), *range(tokens - 40, tokens)) if 0 <= t < tokens]
    for i, (x, y, dy) in enumerate(((q, qo, dq), (k, ko, dk))):
        w = U.f64(weight[i])
        want, mag = dense.rotary(U.f64(x[some]), w, some, U.f64(freq), eps=1e-6)
        U.near(y[some], want, mag, 40, f"heads {i}")
        want = dense.rotary_backward(U.f64(x[some]), w, U.f64(d[i][some]), some, U.f64(freq), eps=1e-6)
        U.near(dy[some], want[0], want[1], 64, f"gradients {i}")
        angle = torch.arange(tokens, device="cuda").double()[:, None, None] * freq.double()
        a, b = d[i][..., :dim // 2].double(), d[i][..., dim // 2:].double()
        u = torch.cat([a * angle.cos() + b * angle.sin(), b * angle.cos() - a * angle.sin()], dim=-1)
        size = (a.abs() + b.abs()).repeat(1, 1, 2)
        unit = x.double() / (x.double().square().mean(dim=-1, keepdim=True) + 1e-6).sqrt()
        sums, mags = (u * unit).sum(dim=(0, 1)).cpu().numpy(), (size * unit.abs()).sum(dim=(0, 1)).cpu().numpy()
        # a thread's items (256 workgroups of 512 threads for a column), their groups, the workgroups' sums
        U.near(dw[i], sums, mags, 64 + tokens * heads // 16 + 512 + 128, f"weight {i}")
