"""The gradients of SwiGLU over more tiles than there are compute units: a
workgroup goes on to further ones."""

import numpy as np
import pytest
import torch

from oracle import dense
from tests import block_util as U
from tests import dense_util as D
from tests.test_gpu_dense import _swiglu_backward

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("grads", [False, True])
def test_swiglu_backward_of_many_tiles(dtype, grads):
    T, C = 600, 8320                             # 5 x 65 tiles, the last row of them ragged
    g = D.generator(T)
    both = D.randn(g, T, 2 * C, scale=2.0, dtype=dtype)
    x, up, dh = both[:, :C], both[:, C:], D.randn(g, T, C, scale=1e-2, dtype=dtype)
    o = _swiglu_backward(x, up, dh, grads=grads)
    dx, dx_mag, dup, dup_mag = dense.swiglu_backward(U.f64(x), U.f64(up), U.f64(dh))
    n = 16                                       # exp, sums, quotient and four products
    if grads:
        U.near(o["dx"], dx, dx_mag, n, "dx")
        U.near(o["dup"], dup, dup_mag, n, "dup")
    v, mag = np.concatenate([dx, dup], axis=1), np.concatenate([dx_mag, dup_mag], axis=1)
    D.check_codes(o["q"], o["q_sf"], dense.rows_quotients(v, mag), n, "q")
    D.check_codes(o["qt"], o["qt_sf"], dense.transposed_quotients(v, mag), n, "qt")
    assert bool((o["qt"][:, T:] == 0).all())
