"""The float64 reference of the operators around the layer: gradients against
central differences, the selection against a search over subsets, and closed
forms."""

import itertools

import numpy as np
import pytest

from oracle import block


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


@pytest.mark.parametrize("kind", ["none", "token", "channel", "full"])
@pytest.mark.parametrize("post", [False, True])
def test_norm_gradients_match_differences(kind, post):
    rng = np.random.default_rng(len(kind) + 10 * post)
    T, H = 3, 16
    h, y = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    gate = {"none": None, "token": rng.standard_normal(T), "channel": rng.standard_normal(H),
            "full": rng.standard_normal((T, H))}[kind]
    pw, qw = (rng.standard_normal(H) if post else None), rng.standard_normal(H)
    dr, dn = rng.standard_normal((T, H)), rng.standard_normal((T, H))

    def loss():
        o = block.norm(h, y, gate, kind, pw, qw, 0.75, 1e-3, 1e-3)
        return (o["r"] * dr).sum() + (o["n"] * dn).sum()

    r = block.norm(h, y, gate, kind, pw, qw, 0.75, 1e-3, 1e-3)["r"]
    g = block.norm_backward(r, dr, dn, y, gate, kind, pw, qw, 0.75, 1e-3, 1e-3)
    _close(g["dh"], _diff(loss, h))
    _close(g["dy"], _diff(loss, y))
    _close(g["dpre"], _diff(loss, qw))
    if post:
        _close(g["dpost"], _diff(loss, pw))
    if gate is not None:
        _close(g["dgate"], _diff(loss, gate))


def test_norm_of_a_constant_row_and_its_codes():
    o = block.norm(np.full((1, 256), -3.0), pre=np.ones(256))
    assert np.allclose(o["n"], -1.0) and np.allclose(o["q_sf"], 1 / 448) and np.allclose(o["q"], -448.0)
    o = block.norm(np.zeros((1, 128)), pre=np.ones(128), pre_eps=1e-6)
    assert not o["q_sf"].any() and not o["q"].any()


def test_router_logits_gradients_match_differences():
    rng = np.random.default_rng(2)
    x, w, d = rng.standard_normal((4, 8)), rng.standard_normal((3, 8)), rng.standard_normal((4, 3))
    g = block.router_logits_backward(d, x, w)
    loss = lambda: (block.router_logits(x, w)[0] * d).sum()   # noqa: E731
    _close(g["dx"], _diff(loss, x))
    _close(g["dw"], _diff(loss, w))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 1), (3, 2, 1), (3, 2, 2)])
def test_selection_maximises_over_subsets(score, groups, kept, top):
    rng = np.random.default_rng(5)
    T, E, k = 20, 12, 3
    l, bias = rng.standard_normal((T, E)), rng.standard_normal(E) * 0.1
    idx, w = block.router_topk(l, k, score, bias, groups=groups, topk_groups=kept, group_top=top, scale=2.0)
    s = block.scores(l, score)
    size = E // groups
    for t in range(T):
        c = s[t] + bias
        best_groups = max(itertools.combinations(range(groups), kept),
                          key=lambda gs: sum(sum(sorted(c[g * size:(g + 1) * size])[-top:]) for g in gs))
        allowed = [e for e in range(E) if e // size in best_groups]
        want = max(itertools.combinations(allowed, k), key=lambda es: sum(c[list(es)]))
        assert sorted(idx[t]) == sorted(want)
        assert np.all(np.diff(c[idx[t]]) <= 0)
        assert np.allclose(w[t], 2.0 * s[t, idx[t]] / s[t, idx[t]].sum())


def test_selection_of_ties_masked_experts_and_masked_tokens():
    l = np.zeros((3, 4))
    l[1, :3] = -np.inf
    l[1, 3] = -5.0
    idx, w = block.router_topk(l, 2, "softmax", mask=[1, 1, 0])
    assert idx.tolist() == [[0, 1], [3, -1], [-1, -1]]
    assert np.allclose(w, [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0]])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_router_gradients_match_differences(score, renormalize):
    rng = np.random.default_rng(7)
    T, E, k = 6, 5, 2
    l = rng.standard_normal((T, E))
    cu, mask = [0, 2, 2, 5], np.array([1, 1, 1, 0, 1, 1])
    idx, _ = block.router_topk(l, k, score, mask=mask, renormalize=renormalize)
    dw, dloss = rng.standard_normal((T, k)), rng.standard_normal(2)
    o = block.balance_loss(l, idx, score, cu, mask, 0.3, 0.2)

    def loss():
        s = block.scores(l, score)
        at = np.where(idx < 0, 0, idx)
        w = np.where(idx < 0, 0.0, np.take_along_axis(s, at, axis=1))
        if renormalize:
            total = w.sum(axis=1, keepdims=True)
            w = w / np.where(total == 0, 1.0, total)
        return (1.5 * w * dw).sum() + (block.balance_loss(l, idx, score, cu, mask, 0.3, 0.2)["loss"] * dloss).sum()

    got, _ = block.router_backward(l, score, idx, dw, renormalize, 1.5, mask, dloss, cu, o["counts"], o["tokens"], k,
                                   0.3, 0.2)
    _close(got, _diff(loss, l))


def test_even_routing_has_balance_loss_one_and_counts_by_hand():
    E, k, T = 4, 2, 8
    idx = np.array([[t % E, (t + 1) % E] for t in range(T)])
    o = block.balance_loss(np.zeros((T, E)), idx, "softmax", balance_coeff=1.0, z_coeff=1.0)
    assert np.isclose(o["loss"][0], 1.0) and np.isclose(o["loss"][1], np.log(E) ** 2)
    assert o["counts"].tolist() == [[4, 4, 4, 4]] and o["tokens"].tolist() == [8, 8, 1]
    o = block.balance_loss(np.zeros((T, E)), idx, "sigmoid", cu=[0, 3, 3, 4], balance_coeff=1.0)
    assert o["counts"].tolist() == [[1, 2, 2, 1], [0, 0, 0, 0], [1, 0, 0, 1]] and o["tokens"].tolist() == [3, 0, 1, 4, 2]
