"""The float64 reference of the dense path: sums written out, gradients against
central differences, and closed forms."""

import math

import numpy as np
import pytest

from oracle import dense


def _diff(f, v, h=1e-6):
    """Central differences of a scalar function of an array."""
    out = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        old = v[i]
        v[i] = old + h
        up = f()
        v[i] = old - h
        out[i] = (up - f()) / (2 * h)
        v[i] = old
    return out


def _close(got, want, tol=1e-7):
    # central differences of step 1e-6: truncation ~ h^2, cancellation ~ 1e-16 / h
    scale = max(np.abs(want).max(), 1e-3)
    assert np.abs(got - want).max() <= tol * scale, np.abs(got - want).max() / scale


@pytest.mark.parametrize("by_rows", [False, True])
def test_product_is_the_sum_of_its_definition(by_rows):
    rng = np.random.default_rng(3)
    m, n, k = 3, 136, 256
    a, b, add = rng.integers(-9, 10, (m, k)), rng.integers(-9, 10, (n, k)), rng.standard_normal((m, n))
    a_sf, b_sf = rng.random((m, 2)), rng.random((n if by_rows else 2, 2))
    out, mag, cut = dense.product(a, a_sf, b, b_sf, by_rows, add)
    for i, j in ((0, 0), (2, 127), (1, 128), (2, 135)):
        want, size, largest = add[i, j], abs(add[i, j]), 0.0
        for s in range(2):
            scale = a_sf[i, s] * b_sf[j if by_rows else j // 128, s]
            terms = [scale * a[i, c] * b[j, c] for c in range(128 * s, 128 * s + 128)]
            want, size, largest = want + sum(terms), size + sum(map(abs, terms)), largest + max(map(abs, terms))
        assert math.isclose(out[i, j], want, rel_tol=1e-12) and math.isclose(mag[i, j], size, rel_tol=1e-12)
        assert cut[i, j] >= 64 * 2.0 ** -16 * largest


def test_quotients_reach_the_largest_code_and_scale_back():
    rng = np.random.default_rng(4)
    v = rng.standard_normal((200, 384))
    v[5, 128:256] = 0.0
    rows, cols, blocks = dense.rows_quotients(v), dense.transposed_quotients(v), dense.block_quotients(v)
    assert rows["sf"].shape == (200, 3) and cols["sf"].shape == (384, 2) and blocks["sf"].shape == (2, 3)
    assert rows["sf"][5, 1] == 0.0 and (rows["q"][5, 128:256] == 0.0).all()
    top = np.abs(rows["q"]).reshape(200, 3, 128).max(axis=2)
    assert np.allclose(np.delete(top.ravel(), 5 * 3 + 1), 448.0, rtol=1e-14)
    assert np.allclose(dense.wide_scales(rows["sf"], 200, True) * rows["q"], v, rtol=1e-14, atol=0)
    assert np.allclose((dense.wide_scales(cols["sf"], 384, True) * cols["q"])[:, :200], v.T, rtol=1e-14, atol=0)
    assert (cols["q"][:, 200:] == 0.0).all()
    assert np.allclose(dense.wide_scales(blocks["sf"], 200, False) * blocks["q"], v, rtol=1e-14, atol=0)
    assert math.isclose(blocks["sf"][1, 2], np.abs(v[128:, 256:]).max() / 448.0)


@pytest.mark.parametrize("clamp", [0.0, 1.25])
def test_swiglu_gradients_match_differences(clamp):
    rng = np.random.default_rng(5)
    x, up, dh = (rng.standard_normal((2, 40)) for _ in range(3))
    loss = lambda: (dense.swiglu(x, up, clamp) * dh).sum()   # noqa: E731
    dx, _, dup, _ = dense.swiglu_backward(x, up, dh, clamp)
    _close(dx, _diff(loss, x))
    _close(dup, _diff(loss, up))


def test_swiglu_at_known_points():
    assert dense.swiglu(np.array([0.0, math.log(3.0), -math.log(3.0)]), np.array([5.0, 4.0, 4.0])).tolist() == pytest.approx(
        [0.0, 3.0 * math.log(3.0), -math.log(3.0)], rel=1e-14)
    dx, _, dup, _ = dense.swiglu_backward(np.zeros(1), np.array([4.0]), np.array([3.0]))
    assert dx.tolist() == [6.0] and dup.tolist() == [0.0]
    assert np.isfinite(dense.swiglu(np.array([-1e4, 1e4]), np.ones(2))).all()


@pytest.mark.parametrize("weight", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("start,half", [(0, 8), (4, 3), (0, 0)])
def test_rotary_gradients_match_differences(weight, interleaved, start, half):
    rng = np.random.default_rng(half + 10 * start)
    x, w, d = rng.standard_normal((2, 3, 16)), (rng.standard_normal(16) if weight else None), rng.standard_normal((2, 3, 16))
    args = dict(positions=np.array([3, 100]), inv_freq=rng.random(half), start=start, interleaved=interleaved, eps=1e-3, scale=1.25)
    loss = lambda: (dense.rotary(x, w, **args)[0] * d).sum()   # noqa: E731
    dx, _, dw, _ = dense.rotary_backward(x, w, d, **args)
    _close(dx, _diff(loss, x))
    if weight:
        _close(dw, _diff(loss, w))


def test_rotary_turns_pairs_by_their_angle():
    # angle 1/2 turn, 1/4 turn; the halves' pairs are (0, 2), (1, 3), the neighbours' (0, 1), (2, 3)
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    args = dict(positions=[1], inv_freq=[math.pi, math.pi / 2], start=0)
    assert dense.rotary(x, None, **args)[0].ravel().tolist() == pytest.approx([-1.0, -4.0, -3.0, 2.0, 9.0], abs=1e-14)
    assert dense.rotary(x, None, interleaved=True, **args)[0].ravel().tolist() == pytest.approx([-1.0, -2.0, -4.0, 3.0, 9.0], abs=1e-14)


def test_scores_depend_on_the_distance_of_positions_alone():
    rng = np.random.default_rng(8)
    q, k = rng.standard_normal((1, 1, 32)), rng.standard_normal((1, 1, 32))
    f = dense.frequencies(32, 10000.0)[0]
    turn = lambda v, p: dense.rotary(v, None, [p], f)[0].ravel()   # noqa: E731
    scores = [turn(q, p + 17) @ turn(k, p) for p in (0, 5, 1000, -40)]
    assert np.allclose(scores, scores[0], rtol=1e-10)


def test_norm_of_a_constant_head():
    out = dense.rotary(np.full((1, 1, 8), -3.0), np.arange(8.0), [0], [])[0]
    assert np.allclose(out.ravel(), -np.arange(8.0))


def test_frequencies_by_parts_between_the_two_plain_forms():
    plain, one = dense.frequencies(64, 10000.0)
    slow, _ = dense.frequencies(64, 10000.0, 8.0)
    parts, scale = dense.frequencies(64, 10000.0, 8.0, 4096.0, 32.0, 1.0)
    assert plain[0] == 1.0 and one == 1.0 and math.isclose(plain[16], 0.01)
    assert np.allclose(np.array(plain) / 8.0, slow)
    assert math.isclose(scale, 0.1 * math.log(8.0) + 1.0)
    turns = [4096.0 * f / (2 * math.pi) for f in plain]
    for i in range(32):
        assert slow[i] * (1 - 1e-12) <= parts[i] <= plain[i] * (1 + 1e-12)
        if turns[i] > 60.0:
            assert parts[i] == plain[i]
        if turns[i] < 0.5:
            assert math.isclose(parts[i], slow[i])
