"""The product's kernels over long loops: every kind of tile, whole and in
parts, with more steps to a part than two rounds of scales last for and a number
that is no multiple of theirs, rows and columns left over, and what is added.
tests/test_product_plan.py holds the sizes to the kinds."""

import pytest
import torch

from tests import block_util as U
from tests import dense_util as D

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32

# (m, k, n): kind and parts
CASES = {
    BF16: {
        (1, 7168, 18432): ("FEW", 1), (1, 6400, 16456): ("FEW", 1), (2, 3200, 4360): ("FEW", 1), (4, 3200, 16400): ("FEW", 1),
        (7, 2176, 4360): ("FEW", 1), (3, 5760, 520): ("FEW", 1), (9, 4736, 1000): ("FEW", 1),
        (17, 2304, 72): ("LOW", 1), (11, 8704, 40): ("LOW", 4), (1, 2304, 12376): ("STRIP", 1), (8, 13952, 2128): ("STRIP", 4),
        (33, 2432, 8304): ("DEEP", 1), (35, 10624, 2152): ("DEEP", 4), (347, 2304, 5400): ("PAIR", 1), (1502, 2176, 1320): ("PAIR", 1),
        (1, 9472, 16424): ("HALF", 1), (33, 8960, 4328): ("HALF", 4), (193, 2432, 16912): ("MID", 1), (193, 2304, 17624): ("MID", 1),
        (136, 2176, 17248): ("TALL", 1), (143, 8704, 5496): ("TALL", 4), (65, 2304, 16800): ("LONG", 1), (68, 8832, 5640): ("LONG", 4),
        (388, 2304, 16464): ("WIDE", 1), (513, 2176, 13624): ("WIDE", 1), (203, 4864, 16800): ("WIDE", 2)},
    F32: {
        (4, 4480, 19160): ("FEW", 1), (1, 2176, 18440): ("FEW", 1), (15, 8064, 3832): ("FEW", 1),
        (17, 2304, 72): ("LOW", 1), (1, 10752, 1048): ("LOW", 4), (10, 2304, 13152): ("DEEP", 1), (33, 4352, 4560): ("DEEP", 2),
        (65, 2304, 8224): ("PAIR", 1), (65, 2304, 16800): ("MID", 1), (276, 4992, 10760): ("MID", 2),
        (193, 2304, 17624): ("WIDE", 1), (66, 8832, 8352): ("WIDE", 4), (65, 4736, 17184): ("WIDE", 2)},
}


def _values(codes, sf, scale):
    """The operand in float64, and per 64 columns its rows' largest magnitude."""
    if scale == "block":
        sf = sf.repeat_interleave(128, dim=0)[:codes.shape[0]]
    v = codes.view(torch.float8_e4m3fn).double() * sf.double().repeat_interleave(128, dim=1)
    return v, v.abs().view(v.shape[0], -1, 64).amax(dim=2)


def _reference(a, a_sf, b, b_sf, scale):
    """As oracle/dense.py's product (out, mag, cut), in float64 on the GPU: its sums are long for the CPU."""
    (va, ta), (vb, tb) = _values(a, a_sf, "row"), _values(b, b_sf, scale)
    out = (va @ vb.t()).cpu().numpy()
    mag = (va.abs_() @ vb.abs_().t()).cpu().numpy()
    return out, mag, (ta @ tb.t()).cpu().numpy() * (64 * 2.0 ** -16)


@pytest.mark.parametrize("scale", ["block", "row"])
def test_reference_is_the_oracle_s(scale):
    g = D.generator(1)
    a, a_sf = D.operand(g, 5, 512)
    b, b_sf = D.operand(g, 136, 512, scale)
    for got, want in zip(_reference(a, a_sf, b, b_sf, scale), D.reference(a, a_sf, b, b_sf, scale)):
        # sums of 512 terms in another order
        assert (abs(got - want) <= 512 * 2.0 ** -52 * D.reference(a, a_sf, b, b_sf, scale)[1] + 1e-300).all()


@pytest.mark.parametrize("scale", ["block", "row"])
@pytest.mark.parametrize("out_type,size", [(t, s) for t, sizes in CASES.items() for s in sizes], ids=lambda v: "x".join(map(str, v)) if isinstance(v, tuple) else str(v)[6:])
def test_product_over_many_steps(out_type, size, scale):
    m, k, n = size
    g = D.generator(m + k + n)
    a, a_sf = D.operand(g, m, k)
    b, b_sf = D.operand(g, n, k, scale)
    want, mag, cut = _reference(a, a_sf, b, b_sf, scale)
    buf = torch.full((m + 1, n), 7.0, dtype=out_type, device="cuda")
    out = buf[:m]
    D.product(a, a_sf, b, b_sf, out, scale)
    D.check_product(out, a, a_sf, b, b_sf, scale, ref=(want, mag, cut), label="alone")
    add = D.randn(g, m, n, scale=30.0, dtype=out_type)
    ref = (want + U.f64(add), mag + abs(U.f64(add)), cut)
    D.product(a, a_sf, b, b_sf, out, scale, add)
    D.check_product(out, a, a_sf, b, b_sf, scale, ref=ref, label="added to")
    first = out.clone()
    out.copy_(add)
    D.product(a, a_sf, b, b_sf, out, scale, out)
    assert torch.equal(out, first)
    assert bool((buf[m] == 7).all())
