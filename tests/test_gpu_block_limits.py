"""GPU tests of the operators around the layer where rounding or float32's range
decides."""

import numpy as np
import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from oracle import block, codecs
from tests import block_util as U
from tests.test_gpu_block import _gen, _np, _topk

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# ---- codes of the norm ---------------------------------------------------------------

def _next_to_ties(blocks, seed):
    """Blocks of 128 float32 values next to ties of E4M3, where the product with
    the reciprocal of amax / 448 rounds to another code than the quotient.  Also
    their scales, the quotients' codes and how many of the products' differ."""
    rng = np.random.default_rng(seed)
    grid = codecs.e4m3_decode(np.arange(127, dtype=np.uint8)).astype(np.float64)
    ties = (grid[1:] + grid[:-1]) / 2
    out, scales, differ = [], [], 0
    for _ in range(blocks):
        amax = np.float32(rng.uniform(1.0, 2.0) * 2.0 ** rng.integers(-3, 4))
        sf = amax / np.float32(448.0)
        near = (ties * np.float64(sf)).astype(np.float32)
        cand = np.concatenate([near] + [(near.view(np.int32) + d).view(np.float32) for d in (-3, -2, -1, 1, 2, 3)])
        cand = cand[cand < amax]
        other = (codecs.e4m3_encode_rne((cand * (np.float32(1.0) / sf)).astype(np.float64))
                 != codecs.e4m3_encode_rne((cand / sf).astype(np.float64)))
        pick = np.concatenate([cand[other], rng.permutation(cand[~other])])[:127]
        differ += min(int(other.sum()), 127)
        b = np.concatenate([[amax], pick]).astype(np.float32) * rng.choice([-1.0, 1.0], 128).astype(np.float32)
        out.append(b)
        scales.append(sf)
    v, s = np.stack(out), np.array(scales, np.float32)
    return v.reshape(-1), s, codecs.e4m3_encode_rne((v / s[:, None]).astype(np.float64)).reshape(-1), differ


@pytest.mark.parametrize("H", [128, 1024, 8192])
def test_codes_are_those_of_the_quotient(H):
    # ones as the stream and no epsilon: the pre-norm is 1 and n the weight itself
    w, sf, want, differ = _next_to_ties(H // 128, H)
    assert differ >= H // 128
    T = 3
    h = torch.ones(T, H, dtype=BF16, device="cuda")
    q, q_sf = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, H // 128, device="cuda")
    B.mega_moe_norm(B.make_args(B.mega_moe_norm_args, num_tokens=T, hidden=H, stream_type=B.MEGA_MOE_BF16,
                                weight_type=B.MEGA_MOE_F32, residual_scale=1.0, h=h, q=q, q_sf=q_sf,
                                pre_weight=torch.from_numpy(w).cuda()), U.current_stream())
    for t in range(T):
        assert np.array_equal(_np(q_sf)[t], sf)
        assert np.array_equal(_np(q)[t], want), int((_np(q)[t] != want).sum())


def test_codes_keep_the_sign_of_zero_and_blocks_of_an_infinite_scale():
    H = 384
    w = np.ones(H, np.float32)
    w[:128:2] = -0.0                              # zeros of both signs beside ones
    w[1:128:4] = 0.0
    w[128:256] = -0.0                             # a block of zeros
    w[256] = np.inf                               # n / inf is 0, inf / inf is not a number
    h = torch.ones(1, H, dtype=BF16, device="cuda")
    q, q_sf = torch.empty(1, H, dtype=torch.uint8, device="cuda"), torch.empty(1, H // 128, device="cuda")
    B.mega_moe_norm(B.make_args(B.mega_moe_norm_args, num_tokens=1, hidden=H, stream_type=B.MEGA_MOE_BF16,
                                weight_type=B.MEGA_MOE_F32, residual_scale=1.0, h=h, q=q, q_sf=q_sf,
                                pre_weight=torch.from_numpy(w).cuda()), U.current_stream())
    got, v = _np(q)[0], U.codes(q)[0]
    assert np.array_equal(got[:128] == 0x80, np.signbit(w[:128])) and np.all(v[3:128:4] == 448.0)
    assert not v[128:256].any() and _np(q_sf)[0, 1] == 0.0
    assert np.isnan(v[256]) and not v[257:].any() and np.isinf(_np(q_sf)[0, 2])


# ---- scores near the smallest floats ---------------------------------------------------

# where a row's logits lie: ordinary, on both sides of where sums of sigmoids get
# too small for their reciprocals, and where every sigmoid is below the smallest float
BASES = np.array([0.0, -30.0, -54.0, -56.0, -70.0, -87.0, -88.5, -91.0, -95.0, -100.0, -104.0, -120.0, -300.0], np.float32)


def _low_rows(T, E, k, seed, bf16=False):
    """Logits around BASES in turn, and k different experts of every token."""
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((T, E)) + BASES[np.arange(T) % len(BASES), None]).astype(np.float32)
    idx = np.argsort(rng.random((T, E)), axis=1)[:, :k].astype(np.int32)
    l = torch.from_numpy(l).cuda()
    return (l.to(BF16) if bf16 else l), idx


def _losses(logits, idx, score, cu, z_coeff):
    T, E = logits.shape
    n = 1 if cu is None else len(cu) - 1
    o = dict(loss=torch.full((2,), 7.0, device="cuda"), counts=torch.empty(n, E, dtype=torch.int32, device="cuda"),
             tokens=torch.empty(n + 2, dtype=torch.int32, device="cuda"), probs=torch.full((n, E), 7.0, device="cuda"))
    a = B.make_args(B.mega_moe_balance_loss_args, num_tokens=T, num_experts=E, num_topk=idx.shape[1],
                    logits_type=U.TYPE[logits.dtype], score=U.SCORE[score], num_sequences=0 if cu is None else n,
                    balance_coeff=0.5, z_coeff=z_coeff, logits=logits, topk_idx=torch.from_numpy(idx).cuda(),
                    cu_seqlens=None if cu is None else torch.tensor(cu, dtype=torch.int32).cuda(), **o)
    B.set_args(a, **U.workspace(B.mega_moe_balance_loss_workspace_bytes(a)))
    B.mega_moe_balance_loss(a, U.current_stream())
    torch.cuda.synchronize()
    return o


LOW = [(13, 4, 1, False), (26, 16, 2, False), (65, 30, 3, True), (100, 64, 4, False), (60, 100, 6, False), (130, 256, 8, False),
       (39, 500, 4, True), (27, 1000, 8, False)]


@pytest.mark.parametrize("T,E,k,bf16", LOW)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("z", [0.0, 0.25])
def test_balance_loss_of_low_logits(T, E, k, bf16, score, z):
    logits, idx = _low_rows(T, E, k, T + E, bf16)
    for cu in (None, list(range(T + 1))):            # all tokens together, and each for itself
        o = _losses(logits, idx, score, cu, z)
        want = block.balance_loss(U.f64(logits), idx, score, cu, None, 0.5, z)
        assert np.array_equal(_np(o["counts"]), want["counts"])
        # p: 32 roundings and E / 64 + 6 adds; then at most T adds of positive terms,
        # E of them in the loss, and one per sequence
        adds = 32 + E // 64 + T
        U.near(o["probs"], want["probs"], want["probs"], adds, "probs")
        U.near(o["loss"], want["loss"], want["loss_mag"], adds + E + T, "loss")
    assert np.allclose(_np(o["probs"]).sum(axis=1), 1.0, atol=1e-5)      # every token is one sequence's all


def _gradient(logits, idx, score, dw=None, renormalize=True, scale=1.5, losses=None, z=0.0):
    """dlogits and the reference's, of the weights' gradient, the losses' or both."""
    T, E = logits.shape
    k = idx.shape[1]
    d = torch.full((T, E), 7.0, device="cuda")
    f = dict(num_tokens=T, num_experts=E, num_topk=k, logits_type=U.TYPE[logits.dtype], score=U.SCORE[score], logits=logits,
             dlogits=d)
    want = {}
    if dw is not None:
        f.update(topk_idx=torch.from_numpy(idx).cuda(), dweights=dw, renormalize=int(renormalize), weight_scale=scale)
        want.update(idx=idx, dweights=U.f64(dw), renormalize=renormalize, scale=scale)
    if losses is not None:
        ref = block.balance_loss(U.f64(logits), idx, score, None, None, 0.5, z)
        f.update(dloss=losses, counts=torch.from_numpy(ref["counts"].astype(np.int32)).cuda(),
                 tokens=torch.from_numpy(ref["tokens"].astype(np.int32)).cuda(), balance_coeff=0.5, z_coeff=z)
        want.update(dloss=U.f64(losses), counts=ref["counts"], tokens=ref["tokens"], k=k, balance_coeff=0.5, z_coeff=z)
    B.mega_moe_router_backward(B.make_args(B.mega_moe_router_backward_args, **f), U.current_stream())
    torch.cuda.synchronize()
    return (d, *block.router_backward(U.f64(logits), score, **want))


@pytest.mark.parametrize("T,E,k,bf16", LOW)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("z", [0.0, 0.25])
def test_gradient_of_the_losses_of_low_logits(T, E, k, bf16, score, z):
    logits, idx = _low_rows(T, E, k, T + E + 1, bf16)
    d, want, mag = _gradient(logits, idx, score, losses=_gen(T)(2), z=z)
    # scores: 32 roundings and E / 64 + 6 adds; the sums over experts the same again
    U.near(d, want, mag, 2 * (48 + E // 64), "dlogits")


# ---- quotients of small scores ------------------------------------------------------------

def _below_the_top(T, E, k, seed):
    """Rows of which one expert has nearly all of the softmax, and k others: their
    scores are next to or below the smallest float."""
    rng = np.random.default_rng(seed)
    l = (rng.standard_normal((T, E)) - rng.choice([20.0, 60.0, 87.0, 95.0, 100.0], (T, 1))).astype(np.float32)
    l[:, 0] = 0.0
    idx = np.argsort(rng.random((T, E - 1)), axis=1)[:, :k].astype(np.int32) + 1
    return torch.from_numpy(l).cuda(), idx


SLOTS = [(26, 4, 1), (39, 8, 2), (52, 40, 5), (65, 64, 8), (40, 256, 8), (2100, 100, 6), (30, 100, 70), (26, 600, 100)]


@pytest.mark.parametrize("T,E,k", SLOTS)
@pytest.mark.parametrize("renormalize", [True, False])
def test_weights_of_small_scores(T, E, k, renormalize):
    # sigmoids of low logits; the order is that of the logits, and of scores with a
    # bias that moves only the first expert
    first = torch.zeros(E, device="cuda")
    first[0] = -10.0
    low, _ = _low_rows(T, E, k, T + 2)
    top, _ = _below_the_top(T, E, k, T + 3)
    for logits, score, bias in ((low, "sigmoid", None), (low, "sigmoid", first), (top, "softmax", first),
                                (top, "softmax", None)):
        if bias is not None and k == E:
            continue
        # slots beyond what float32 can tell are not asked for: the indices are
        # checked elsewhere, the weights are those of the indices given
        idx, w = _topk(logits, k, score, bias, renormalize=renormalize)
        at = _np(idx)
        assert at.min() >= 0 and all(len(set(r)) == k for r in at.tolist())
        s = np.take_along_axis(block.scores(U.f64(logits), score), at.astype(np.int64), axis=1)
        want = 2.5 * s / (s.sum(axis=1, keepdims=True) if renormalize else 1.0)
        # exp and the division carry a few roundings, and the difference to the
        # row's largest logit half a step of up to 128
        U.near(w, want, want, 32 + 128 + E // 64 + k, f"{score} {bias is not None}")


# logits, score, bias: every expert that is taken has a score below the smallest normal float
ONLY = [([0.0, -95.0], "softmax", [-10.0, 0.0]), ([-95.0, -110.0], "sigmoid", None), ([-88.0, -120.0], "sigmoid", [0.0, -1.0]),
        ([0.0, -100.0, -103.0], "softmax", [-10.0, 0.0, -1.0])]


@pytest.mark.parametrize("logits,score,bias", ONLY)
def test_weight_of_the_only_slot_is_the_scale(logits, score, bias):
    idx, w = _topk(torch.tensor([logits], device="cuda"), 1, score, None if bias is None else torch.tensor(bias, device="cuda"))
    assert w.tolist() == [[2.5]], (idx.tolist(), w.tolist())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_large_weight_scale_over_a_small_sum(score):
    # scale / sum is beyond float32 in some rows, the weights in none
    T, E, k = 9, 32, 3
    r = _gen(5)
    l = r(T, E) - 6.0
    l[:, 0] = 3.0
    bias = torch.zeros(E, device="cuda")
    bias[0] = -10.0
    scale = 1e37
    idx, w = _topk(l, k, score, bias, scale=scale)
    s = np.take_along_axis(block.scores(U.f64(l), score), _np(idx).astype(np.int64), axis=1)
    want = float(np.float32(scale)) * s / s.sum(axis=1, keepdims=True)
    assert float(np.float32(scale)) / s.sum(axis=1).min() > 3.5e38
    U.near(w, want, want, 64, "weights")


@pytest.mark.parametrize("T,E,k", SLOTS)
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_of_the_weights_of_small_scores(T, E, k, renormalize):
    r = _gen(T + E)
    for (logits, idx), score in ((_low_rows(T, E, k, T + 4), "sigmoid"), (_below_the_top(T, E, min(k, E - 1), T + 5), "softmax"),
                                 (_low_rows(T, E, k, T + 6), "softmax")):
        dw = r(T, idx.shape[1])
        d, want, mag = _gradient(logits, idx, score, dw, renormalize)
        # as for the weights, twice, and the sums over slots
        U.near(d, want, mag, 2 * (48 + 128 + E // 64) + 2 * k, score)


@pytest.mark.parametrize("logits,score,bias", ONLY)
def test_gradient_of_the_only_weight_is_zero(logits, score, bias):
    l = torch.tensor([logits], device="cuda")
    idx, _ = _topk(l, 1, score, None if bias is None else torch.tensor(bias, device="cuda"))
    d, want, _ = _gradient(l, _np(idx), score, dw=torch.full((1, 1), 3.0, device="cuda"))
    assert not want.any() and np.all(np.abs(_np(d)) <= 2.0 ** -20), d.tolist()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradient_of_a_large_weight_scale_over_a_small_sum(score):
    T, E, k = 9, 32, 3
    r = _gen(6)
    l = r(T, E) - 6.0
    l[:, 0] = 3.0
    idx = (np.arange(T * k).reshape(T, k) % (E - 1) + 1).astype(np.int32)
    scale = float(np.float32(1e37))
    assert scale / np.take_along_axis(block.scores(U.f64(l), score), idx.astype(np.int64), axis=1).sum(axis=1).min() > 3.5e38
    d, want, mag = _gradient(l, idx, score, r(T, k), True, scale)
    U.near(d, want, mag, 128, "dlogits")


# ---- tensors the device does not know ------------------------------------------------------------

def test_a_first_tensor_in_host_memory_is_refused():
    T, H, E, k = 4, 256, 8, 2
    here = dict(device="cuda")
    rows, wide = torch.zeros(T, H, dtype=BF16, **here), torch.zeros(T, E, **here)
    w, out, idx = torch.ones(H, **here), torch.full((T, H), 7.0, dtype=BF16, **here), torch.zeros(T, k, dtype=torch.int32, **here)
    ws = U.workspace(1 << 20)
    calls = [
        (B.mega_moe_norm, B.mega_moe_norm_args, "h", rows, dict(num_tokens=T, hidden=H, weight_type=1, residual_scale=1.0,
                                                               pre_weight=w, n=out)),
        (B.mega_moe_norm_backward, B.mega_moe_norm_backward_args, "dr", rows, dict(num_tokens=T, hidden=H, residual_scale=1.0, dh=out)),
        (B.mega_moe_router_logits, B.mega_moe_router_logits_args, "x", rows, dict(num_tokens=T, hidden=H, num_experts=E, logits=wide,
                                                                                 w=torch.zeros(E, H, dtype=BF16, **here), **ws)),
        (B.mega_moe_router_logits_backward, B.mega_moe_router_logits_args, "dlogits", wide,
         dict(num_tokens=T, hidden=H, num_experts=E, w=torch.zeros(E, H, dtype=BF16, **here), dx=out, **ws)),
        (B.mega_moe_router_topk, B.mega_moe_router_topk_args, "logits", wide,
         dict(num_tokens=T, num_experts=E, num_topk=k, logits_type=1, topk_idx=idx, topk_weights=torch.zeros(T, k, **here))),
        (B.mega_moe_balance_loss, B.mega_moe_balance_loss_args, "loss", torch.zeros(2, **here),
         dict(num_tokens=T, num_experts=E, num_topk=k, logits_type=1, logits=wide, topk_idx=idx,
              counts=torch.zeros(E, dtype=torch.int32, **here), tokens=torch.zeros(3, dtype=torch.int32, **here), **ws)),
        (B.mega_moe_router_backward, B.mega_moe_router_backward_args, "logits", wide,
         dict(num_tokens=T, num_experts=E, num_topk=k, logits_type=1, topk_idx=idx, dweights=torch.zeros(T, k, **here),
              dlogits=torch.zeros(T, E, **here))),
    ]
    for call, cls, first, good, others in calls:
        a = B.make_args(cls, **{first: good}, **others)
        assert call(a, U.current_stream()) == 0, call.__name__
        # aligned as a device's tensor is, in ordinary memory: the refusal is the host's
        host = torch.zeros(good.numel() * good.element_size() + 64, dtype=torch.uint8)
        B.set_args(a, **{first: host.data_ptr() + -host.data_ptr() % 64})
        with pytest.raises(B.MegaMoEError) as ei:
            call(a, U.current_stream())
        assert ei.value.code == B.MEGA_MOE_ERR_INVALID_ARG and "host memory" in B.mega_moe_last_error()
    torch.cuda.synchronize()


# ---- float32 operands of the router's products ------------------------------------------------

def _full(r, *shape):
    """Floats whose 24 bits of mantissa are all in use."""
    v = r(*shape)
    return torch.where(v.abs() < 1e-3, torch.full_like(v, 0.7), v)


def _two_terms(v):
    """What is left of a float32 in two BF16 terms."""
    first = v.to(BF16).float()
    return first + (v - first).to(BF16).float()


# through each of the kernels: 16 x 16 tiles; few, some, many experts, workgroups in
# pairs, K in parts and not
@pytest.mark.parametrize("T,H,E", [(3, 40, 5), (64, 512, 64), (129, 2048, 257), (5003, 1160, 17), (3300, 904, 61),
                                   (1030, 776, 260), (8200, 4104, 130), (515, 1152, 300), (2050, 520, 330)])
def test_logits_of_float32_weights_lose_no_bit(T, H, E):
    # a one in every row of x: the logits are columns of w
    r = _gen(T + H)
    w = _full(r, E, H)
    at = torch.randint(0, H, (T,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(H))
    x = torch.zeros(T, H, dtype=BF16, device="cuda")
    x[torch.arange(T, device="cuda"), at] = 1.0
    logits = torch.full((T, E), 7.0, device="cuda")
    a = B.make_args(B.mega_moe_router_logits_args, num_tokens=T, hidden=H, num_experts=E, weight_type=B.MEGA_MOE_F32, x=x, w=w,
                    logits=logits)
    B.set_args(a, **U.workspace(B.mega_moe_router_logits_workspace_bytes(a)))
    B.mega_moe_router_logits(a, U.current_stream())
    want = w[:, at].t()
    assert (_two_terms(want) != want).float().mean() > 0.5       # two terms would not do
    assert torch.equal(logits, want), int((logits != want).sum())


# one step of 64 k in LDS and two, parts of T and not, rows of dlogits padded and not
BACKWARD = [(3, 40, 5), (64, 512, 64), (129, 2048, 257), (515, 1152, 300), (2050, 640, 72), (8200, 1032, 66), (4100, 2056, 70),
            (1100, 256, 8)]


@pytest.mark.parametrize("T,H,E", BACKWARD)
@pytest.mark.parametrize("wt", [BF16, F32])
def test_dw_loses_no_bit(T, H, E, wt):
    # a one in every column of x: the columns of dw are rows of dlogits
    r = _gen(T + E)
    d = _full(r, T, E)
    at = torch.randint(0, T, (H,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(T))
    x = torch.zeros(T, H, dtype=BF16, device="cuda")
    x[at, torch.arange(H, device="cuda")] = 1.0
    w, dx, dw = r(E, H, dtype=wt), torch.empty(T, H, dtype=BF16, device="cuda"), torch.full((E, H), 7.0, device="cuda")
    a = B.make_args(B.mega_moe_router_logits_args, num_tokens=T, hidden=H, num_experts=E, weight_type=U.TYPE[wt], x=x, w=w,
                    dlogits=d, dx=dx, dw=dw)
    B.set_args(a, **U.workspace(B.mega_moe_router_logits_workspace_bytes(a)))
    B.mega_moe_router_logits_backward(a, U.current_stream())
    want = d[at].t()
    assert (_two_terms(want) != want).float().mean() > 0.5
    assert torch.equal(dw, want), int((dw != want).sum())


def _next_to_bf16_ties(r, *shape):
    """Floats one step of float32 above or below the middle of two BF16 values."""
    v = r(*shape).view(torch.int32) & ~0xffff
    return (v + 0x8000 + torch.where(r(*shape) > 0, 1, -1).to(torch.int32)).view(F32)


@pytest.mark.parametrize("T,H,E", BACKWARD)
@pytest.mark.parametrize("which", ["dlogits", "w"])
def test_dx_of_float32_weights_is_rounded_once(T, H, E, which):
    # dx is one product of a one with a float next to a tie of BF16
    r = _gen(T + E + H)
    d, w = torch.zeros(T, E, device="cuda"), torch.zeros(E, H, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(E)
    if which == "w":
        at = torch.randint(0, E, (T,), device="cuda", generator=g)
        d[torch.arange(T, device="cuda"), at] = 1.0
        w = _next_to_bf16_ties(r, E, H)
        exact = w[at]
    else:
        at = torch.randint(0, E, (H,), device="cuda", generator=g)
        w[at, torch.arange(H, device="cuda")] = 1.0
        d = _next_to_bf16_ties(r, T, E)
        exact = d[:, at]
    dx = torch.empty(T, H, dtype=BF16, device="cuda")
    a = B.make_args(B.mega_moe_router_logits_args, num_tokens=T, hidden=H, num_experts=E, weight_type=B.MEGA_MOE_F32, w=w,
                    dlogits=d, dx=dx)
    B.set_args(a, **U.workspace(B.mega_moe_router_logits_workspace_bytes(a)))
    B.mega_moe_router_logits_backward(a, U.current_stream())
    want = exact.to(BF16)
    assert (_two_terms(exact).to(BF16) != want).float().mean() > 0.2     # two terms would not do
    assert torch.equal(dx, want), int((dx != want).sum())
