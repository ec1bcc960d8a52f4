"""Operands and runs of the dense path's operators for the tests."""

from __future__ import annotations

import numpy as np
import torch

from fp8_mixture_experts_amd import binding as B
from oracle import dense
from tests import block_util as U

BF16, F32 = torch.bfloat16, torch.float32
SCALE = {"block": B.MEGA_MOE_SCALE_BLOCK, "row": B.MEGA_MOE_SCALE_ROW}
# rounding to E4M3: half a step is at most 2^-4 of the value, or 2^-10 (half the smallest step)
E4M3_HALF, E4M3_LEAST = 2.0 ** -4, 2.0 ** -10


def up128(n):
    return -(-n // 128) * 128


def randn(g, *shape, scale=1.0, dtype=F32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def spaced(t, extra, fill=0):
    """The same values in rows `extra` elements further apart, and the whole buffer."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    buf[:, :t.shape[1]] = t
    return buf[:, :t.shape[1]], buf


def operand(g, rows, k, scale="row", spread=0.5):
    """Codes over E4M3's finite values, and scales of mixed sizes."""
    codes = torch.randint(0, 256, (rows, k), generator=g, device="cuda", dtype=torch.int32)
    codes = torch.where((codes & 0x7F) == 0x7F, codes & 0x80, codes).to(torch.uint8)
    n = rows if scale == "row" else up128(rows) // 128
    sf = torch.exp(randn(g, n, k // 128, scale=spread)) * 2.0 ** -8
    return codes, sf


def product_args(a, a_sf, b, b_sf, out, scale, add=None, **more):
    m, k = a.shape
    f = dict(m=m, n=b.shape[0], k=k, b_scale=SCALE[scale], out_type=U.TYPE[out.dtype], a=a, a_sf=a_sf, b=b, b_sf=b_sf, add=add, out=out)
    f.update(more)
    args = B.make_args(B.mega_moe_product_args, **f)
    return B.set_args(args, **U.workspace(B.mega_moe_product_workspace_bytes(args)))


def product(*args, stream=None, **kw):
    B.mega_moe_product(product_args(*args, **kw), U.current_stream() if stream is None else stream)


def reference(a, a_sf, b, b_sf, scale, add=None):
    return dense.product(U.codes(a), U.f64(a_sf), U.codes(b), U.f64(b_sf), scale == "row", None if add is None else U.f64(add))


def check_product(out, a, a_sf, b, b_sf, scale, add=None, label="", ref=None):
    """Every element within its type's half step and float32's roundings (a sum of k products of two
    scales; with a BF16 output what the instruction leaves out)."""
    want, mag, cut = reference(a, a_sf, b, b_sf, scale, add) if ref is None else ref
    k = a.shape[1]
    # products are exact; k additions, the scales' product, their application, `add`
    roundings = k + k // 128 + 4
    if out.dtype == BF16:
        mag = mag + cut / (roundings * U.U)
    U.near(out, want, mag, roundings, label)
    if out.dtype == BF16 and np.linalg.norm(want):
        assert np.linalg.norm(U.f64(out) - want) <= 2.0 ** -8 * np.linalg.norm(want), label


def check_codes(q, sf, want, roundings, label=""):
    """q (bytes) and sf against quotients and scales before rounding: a scale is off by float32's roundings, and
    a code by E4M3's half step of a quotient that both its parts' roundings have moved."""
    U.near(sf, want["sf"], want.get("sf_mag", want["sf"]), roundings + 1, label + " sf")
    got, quot = U.codes(q), want["q"]
    mag = want.get("q_mag", np.abs(quot))
    moved = (2 * roundings + 4) * U.U * (mag + np.abs(quot))
    limit = (1 + E4M3_HALF) * moved + E4M3_HALF * np.abs(quot) + E4M3_LEAST
    # the half step above is that of the largest value of a binade; the codes' own steps are finer where these are smaller
    step = np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(quot) - moved, 2.0 ** -12))), -6.0) - 3.0)
    limit = np.minimum(limit, step + moved)
    bad = ~(np.abs(got - quot) <= limit)
    assert not bad.any(), f"{label}: {int(bad.sum())} codes of {bad.size} outside, at {np.argwhere(bad)[:3].tolist()}"
