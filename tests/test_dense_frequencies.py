"""mega_moe_rotary_frequencies by parts against shares that are written out: the
ramp between both bounds may end behind the last frequency."""

import math

import numpy as np
import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from oracle import dense


def _by_parts(dim, base, length, fast, slow, factor):
    inv, scale = torch.full((dim // 2,), 7.0), torch.zeros(1)
    B.mega_moe_rotary_frequencies(B.make_args(
        B.mega_moe_rotary_frequencies_args, rotary_dim=dim, scaling=B.MEGA_MOE_ROTARY_BY_PARTS, base=base, factor=factor,
        original_length=length, fast_turns=fast, slow_turns=slow, inv_freq=inv, scale=scale))
    return inv.double().numpy(), float(scale)


# the whole indices around both bounds, the upper one at most dim - 1
RAMPS = [(128, 1e4, 4096.0, 32.0, 1.0, 20, 46), (64, 1e4, 131072.0, 32.0, 1.0, 22, 35), (16, 1e4, 32768.0, 32.0, 1.0, 4, 8),
         (128, 1e4, 65536.0, 32.0, 1.0, 40, 65), (64, 500.0, 4096.0, 32.0, 1.0, 15, 34), (16, 1e4, 1e9, 1e6, 1.0, 4, 15)]


@pytest.mark.parametrize("dim,base,length,fast,slow,lo,hi", RAMPS)
@pytest.mark.parametrize("factor", [1.0, 4.0, 40.0])
def test_ramp_goes_from_one_bound_to_the_other(dim, base, length, fast, slow, lo, hi, factor):
    def turns(i):
        return length * base ** (-2.0 * i / dim) / (2 * math.pi)

    assert turns(lo) >= fast > turns(lo + 1)
    assert hi == dim - 1 or turns(hi - 1) > slow >= turns(hi)
    want = []
    for i in range(dim // 2):
        share = 0.0 if i <= lo else 1.0 if i >= hi else (i - lo) / (hi - lo)
        f = base ** (-2.0 * i / dim)
        want.append((1.0 - share) * f + share * f / factor)
    inv, scale = _by_parts(dim, base, length, fast, slow, factor)
    # one rounding to float32 behind float64's
    np.testing.assert_allclose(inv, want, rtol=2.0 ** -24 + 1e-12, atol=0)
    assert abs(scale - (0.1 * math.log(factor) + 1.0)) <= 2.0 ** -24 * scale
    np.testing.assert_allclose(dense.frequencies(dim, base, factor, length, fast, slow)[0], want, rtol=1e-12, atol=0)


@pytest.mark.parametrize("dim,base,length,fast,slow", [(64, 1e4, 4.0, 32.0, 1.0), (16, 1e4, 2 * math.pi * 0.999, 2.0, 1.0),
                                                       (32, 500.0, 100.0, 64.0, 16.0), (16, 1e4, 1e-3, 32.0, 1.0)])
def test_frequencies_that_are_all_slow_are_all_divided(dim, base, length, fast, slow):
    plain = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    assert length * plain[0] / (2 * math.pi) < slow
    want = [f / 8.0 for f in plain]
    np.testing.assert_allclose(_by_parts(dim, base, length, fast, slow, 8.0)[0], want, rtol=2.0 ** -24 + 1e-12, atol=0)
    np.testing.assert_allclose(dense.frequencies(dim, base, 8.0, length, fast, slow)[0], want, rtol=1e-12, atol=0)


def test_frequencies_that_are_all_fast_all_stay():
    # 10^12 positions: the last of 32 makes 10^7 turns
    inv, _ = _by_parts(64, 1e4, 1e12, 32.0, 1.0, 8.0)
    np.testing.assert_allclose(inv, [1e4 ** (-i / 32.0) for i in range(32)], rtol=2.0 ** -24 + 1e-12, atol=0)
