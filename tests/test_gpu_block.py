"""GPU parity of the operators around the layer with the float64 reference:
small and odd sizes, long rows, strides, types, gates, masks that leave a row
empty, ragged and empty sequences."""

import numpy as np
import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from oracle import block, codecs
from tests import block_util as U

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *shape, dtype=F32, scale=1.0: (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


# ---- norm ------------------------------------------------------------------------

# tokens, hidden, stream type, weight type, gate kind, gate type, post, extra elements per row
NORM = [
    (1, 8, BF16, F32, "none", F32, False, 0),
    (1, 7168, BF16, F32, "none", F32, False, 0),
    (3, 128, F32, BF16, "token", BF16, True, 8),
    (5, 136, BF16, BF16, "channel", BF16, True, 0),
    (2, 1000, F32, F32, "full", F32, True, 24),
    (17, 2048, BF16, F32, "full", BF16, False, 128),
    (7, 2056, BF16, F32, "token", F32, True, 0),
    (4, 8192, F32, BF16, "channel", F32, True, 0),
    (3, 8184, BF16, BF16, "channel", F32, False, 8),
    (2, 8192, F32, F32, "full", BF16, True, 0),
    (1030, 384, BF16, F32, "channel", F32, True, 0),
    (577, 4096, F32, F32, "token", F32, False, 0),
    # several rounds of rows, the last of them not full
    (6300, 136, BF16, BF16, "channel", F32, True, 0),
    (2100, 1000, F32, F32, "full", BF16, True, 8),
    (6200, 256, BF16, F32, "token", BF16, False, 0),
]


def _norm_inputs(T, H, stream, wt, kind, gt, post, extra, seed=1):
    r = _gen(seed + 13 * T + H)
    gate_shape = {"none": None, "token": (T,), "channel": (H,), "full": (T, H)}[kind]

    def rows(dtype, scale=1.0):
        v, _ = U.padded(T, H, dtype, extra)
        v.copy_(r(T, H, scale=scale))
        return v

    s = {"h": rows(stream, 1.5), "y": rows(BF16, 0.5), "pre": 1.0 + r(H, dtype=wt, scale=0.1),
         "post": (1.0 + r(H, scale=0.1)).to(wt) if post else None, "gate": None}
    s["pre"] = s["pre"].to(wt)
    if kind == "full":
        s["gate"] = rows(gt)
    elif gate_shape:
        s["gate"] = r(*gate_shape, dtype=gt)
    return s, rows, r


def _norm_fields(T, H, stream, wt, kind, gt, s, extra, scale):
    return dict(num_tokens=T, hidden=H, stream_type=U.TYPE[stream], weight_type=U.TYPE[wt], gate_kind=U.KIND[kind],
                gate_type=U.TYPE[gt], post_eps=1e-6, pre_eps=1e-5, residual_scale=scale, y=s["y"], gate=s["gate"],
                post_weight=s["post"], pre_weight=s["pre"], y_stride=H + extra,
                gate_stride=H + extra if kind == "full" else 0)


# A term of r or n passes through at most 16 roundings, and a row's sum of
# squares through at most 32 sequential adds, 6 over a wave, 15 over waves and
# the mean's few, halved by the square root: under 48 in all.
NORM_ROUNDINGS = 48


@pytest.mark.parametrize("T,H,stream,wt,kind,gt,post,extra", NORM)
def test_norm_matches_the_reference(T, H, stream, wt, kind, gt, post, extra):
    s, rows, _ = _norm_inputs(T, H, stream, wt, kind, gt, post, extra)
    r, r_buf = U.padded(T, H, stream, extra)
    n, n_buf = U.padded(T, H, BF16, extra)
    quant = H % 128 == 0
    q = torch.full((T, H), 3, dtype=torch.uint8, device="cuda") if quant else None
    sf = torch.full((T, H // 128), 3.0, device="cuda") if quant else None
    a = B.make_args(B.mega_moe_norm_args, h=s["h"], r=r, n=n, q=q, q_sf=sf, h_stride=H + extra, r_stride=H + extra,
                    n_stride=H + extra, **_norm_fields(T, H, stream, wt, kind, gt, s, extra, 0.875))
    B.mega_moe_norm(a, U.current_stream())
    torch.cuda.synchronize()
    want = block.norm(U.f64(s["h"]), U.f64(s["y"]), U.f64(s["gate"]), kind, U.f64(s["post"]), U.f64(s["pre"]), 0.875,
                      1e-6, 1e-5)
    U.near(r, want["r"], want["r_mag"], NORM_ROUNDINGS, "r")
    U.near(n, want["n"], want["n_mag"], NORM_ROUNDINGS, "n")
    if quant:
        U.near(sf, want["q_sf"], want["q_sf_mag"], NORM_ROUNDINGS, "q_sf")
        # a code is the nearest to n / q_sf, up to what float32 leaves open
        wide = np.repeat(want["q_sf"], 128, axis=1)
        off = np.abs(U.codes(q) - want["q"])
        step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want["q"]), 2.0 ** -6))) - 3)
        slack = NORM_ROUNDINGS * U.U * 3 * np.divide(want["n_mag"], wide, out=np.zeros_like(wide), where=wide > 0)
        assert np.all(off <= 0.5 * step * (1 + 2.0 ** -20) + slack + 2.0 ** -20)
        assert (q == torch.from_numpy(codecs.e4m3_encode_rne(want["q"])).cuda()).float().mean() >= 0.999
    if extra:
        assert torch.all(r_buf[:, H:] == 7.0) and torch.all(n_buf[:, H:] == 7.0)


def test_norm_alone_in_place_and_with_few_outputs():
    T, H = 9, 640
    r = _gen(3)
    h, w = r(T, H, dtype=BF16), r(H)
    n = torch.empty(T, H, dtype=BF16, device="cuda")
    base = dict(num_tokens=T, hidden=H, stream_type=B.MEGA_MOE_BF16, weight_type=B.MEGA_MOE_F32, pre_eps=1e-6)
    B.mega_moe_norm(B.make_args(B.mega_moe_norm_args, h=h, n=n, pre_weight=w, residual_scale=1.0, **base),
                    U.current_stream())
    want = block.norm(U.f64(h), pre=U.f64(w), pre_eps=1e-6)
    U.near(n, want["n"], want["n_mag"], NORM_ROUNDINGS, "n alone")
    # r only, written over h
    y, stream = r(T, H, dtype=BF16), h.clone()
    B.mega_moe_norm(B.make_args(B.mega_moe_norm_args, h=stream, r=stream, y=y, residual_scale=0.5, **base),
                    U.current_stream())
    want = block.norm(U.f64(h), U.f64(y), scale=0.5)
    U.near(stream, want["r"], want["r_mag"], NORM_ROUNDINGS, "r in place")
    # codes only
    q, sf = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, H // 128, device="cuda")
    B.mega_moe_norm(B.make_args(B.mega_moe_norm_args, h=h, q=q, q_sf=sf, pre_weight=w, residual_scale=1.0, **base),
                    U.current_stream())
    want = block.norm(U.f64(h), pre=U.f64(w), pre_eps=1e-6)
    U.near(sf, want["q_sf"], want["q_sf_mag"], NORM_ROUNDINGS, "q_sf alone")
    assert (q == torch.from_numpy(codecs.e4m3_encode_rne(want["q"])).cuda()).float().mean() >= 0.999


# several rows to a group of threads, each loaded while the one before it is stored
@pytest.mark.parametrize("T,H,stream", [(5000, 640, BF16), (2100, 1032, F32), (777, 7168, BF16)])
def test_norm_and_gradients_in_place_equal_those_apart(T, H, stream):
    r = _gen(T + H)
    h, y, dn, w, gate = r(T, H, dtype=stream), r(T, H, dtype=BF16), r(T, H, dtype=BF16), r(H), r(T, dtype=BF16)
    base = dict(num_tokens=T, hidden=H, stream_type=U.TYPE[stream], weight_type=B.MEGA_MOE_F32, pre_eps=1e-6,
                post_eps=1e-6, residual_scale=0.5, y=y, gate=gate, gate_kind=U.KIND["token"], gate_type=B.MEGA_MOE_BF16,
                post_weight=w, pre_weight=w)
    out = []
    for place in (False, True):
        src = h.clone()
        to, n = src if place else torch.empty_like(h), torch.empty(T, H, dtype=BF16, device="cuda")
        B.mega_moe_norm(B.make_args(B.mega_moe_norm_args, h=src, r=to, n=n, **base), U.current_stream())
        dr = h.clone()
        dh, dy, dgate, dw = dr if place else torch.empty_like(h), torch.empty_like(y), r(T), r(H)
        a = B.make_args(B.mega_moe_norm_backward_args, r=to, dr=dr, dn=dn, dh=dh, dy=dy, dgate=dgate, dpost_weight=dw,
                        **base)
        B.set_args(a, **U.workspace(B.mega_moe_norm_workspace_bytes(a)))
        B.mega_moe_norm_backward(a, U.current_stream())
        out.append((to, n, dh, dy, dgate, dw))
    torch.cuda.synchronize()
    for apart, inside in zip(*out):
        assert torch.equal(apart, inside)


def test_norm_of_zero_tiny_and_not_finite_rows():
    T, H = 6, 256
    h = torch.zeros(T, H, device="cuda")
    h[1] = 1e-30                     # mean of squares underflows: eps alone is left
    h[2] = 1.0
    h[2, 5] = float("nan")
    h[3, :128] = 2.0                 # one block of zeros beside one that is not
    h[4] = 3.0
    h[4, 200] = float("inf")
    h[5] = 1e-38
    w = torch.ones(H, device="cuda")
    n = torch.empty(T, H, dtype=BF16, device="cuda")
    q, sf = torch.empty(T, H, dtype=torch.uint8, device="cuda"), torch.empty(T, H // 128, device="cuda")
    B.mega_moe_norm(B.make_args(B.mega_moe_norm_args, num_tokens=T, hidden=H, stream_type=B.MEGA_MOE_F32,
                                weight_type=B.MEGA_MOE_F32, pre_eps=1e-6, residual_scale=1.0, h=h, n=n, q=q, q_sf=sf,
                                pre_weight=w), U.current_stream())
    n, sf, v = n.float().cpu().numpy(), sf.cpu().numpy(), U.codes(q)
    assert not n[0].any() and not sf[0].any() and not v[0].any()
    assert np.allclose(n[1], 1e-27, rtol=2.0 ** -8) and np.allclose(sf[1], 1e-27 / 448, rtol=1e-5)
    assert np.all(v[1] == 448.0)
    assert np.isnan(n[2]).all() and np.isnan(sf[2]).all() and np.isnan(v[2]).all()
    assert np.allclose(n[3, :128], np.sqrt(2.0), rtol=2.0 ** -8) and not n[3, 128:].any()
    assert np.all(v[3, :128] == 448.0) and not v[3, 128:].any() and sf[3, 1] == 0.0
    # an infinity: 1 / rms is 0, so the finite columns vanish and inf * 0 is NaN
    assert np.isnan(n[4, 200]) and not n[4, :128].any() and np.isnan(sf[4, 1]) and sf[4, 0] == 0.0
    assert np.all(v[5] == 448.0)


@pytest.mark.parametrize("T,H,stream,wt,kind,gt,post,extra", NORM)
def test_norm_backward_matches_the_reference(T, H, stream, wt, kind, gt, post, extra):
    s, rows, _ = _norm_inputs(T, H, stream, wt, kind, gt, post, extra, seed=2)
    dr, dn = rows(stream, 0.1), rows(BF16, 0.1)
    dh, dh_buf = U.padded(T, H, stream, extra)
    dy, dy_buf = U.padded(T, H, BF16, extra)
    dgate = None
    if kind == "full":
        dgate, _ = U.padded(T, H, gt, extra)
    elif kind != "none":
        dgate = torch.full_like(s["gate"], 7.0, dtype=F32)
    dpost = torch.full((H,), 7.0, device="cuda") if post else None
    dpre = torch.full((H,), 7.0, device="cuda")
    a = B.make_args(B.mega_moe_norm_backward_args, r=s["h"], dr=dr, dn=dn, dh=dh, dy=dy, dgate=dgate,
                    dpost_weight=dpost, dpre_weight=dpre, r_stride=H + extra, dr_stride=H + extra, dn_stride=H + extra,
                    dh_stride=H + extra, dy_stride=H + extra, dgate_stride=H + extra if kind == "full" else 0,
                    **_norm_fields(T, H, stream, wt, kind, gt, s, extra, 0.875))
    U.finish_norm_backward(a)
    torch.cuda.synchronize()
    want = block.norm_backward(U.f64(s["h"]), U.f64(dr), U.f64(dn), U.f64(s["y"]), U.f64(s["gate"]), kind,
                               U.f64(s["post"]), U.f64(s["pre"]), 0.875, 1e-6, 1e-5)
    # each norm's backward: two row sums and about 16 roundings a term
    U.near(dh, want["dh"], want["dh_mag"], 2 * NORM_ROUNDINGS, "dh")
    U.near(dy, want["dy"], want["dy_mag"], 4 * NORM_ROUNDINGS, "dy")
    # and sums over the tokens: at most T adds in all
    U.near(dpre, want["dpre"], want["dpre_mag"], 2 * NORM_ROUNDINGS + T, "dpre")
    if post:
        U.near(dpost, want["dpost"], want["dpost_mag"], 4 * NORM_ROUNDINGS + T, "dpost")
    if dgate is not None:
        adds = {"token": NORM_ROUNDINGS, "channel": T, "full": 0}[kind]
        U.near(dgate, want["dgate"], want["dgate_mag"], 4 * NORM_ROUNDINGS + adds, "dgate")
    if extra:
        assert torch.all(dh_buf[:, H:] == 7.0) and torch.all(dy_buf[:, H:] == 7.0)


def test_norm_backward_of_parts():
    # the pre-norm alone; the residual alone, in place; and no tokens
    T, H = 11, 320
    r = _gen(4)
    h, dn, w = r(T, H, dtype=BF16), r(T, H, dtype=BF16), r(H)
    dh, dpre = torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(H, device="cuda")
    base = dict(num_tokens=T, hidden=H, stream_type=B.MEGA_MOE_BF16, weight_type=B.MEGA_MOE_F32, pre_eps=1e-6,
                residual_scale=1.0)
    U.finish_norm_backward(B.make_args(B.mega_moe_norm_backward_args, r=h, dn=dn, dh=dh, dpre_weight=dpre,
                                       pre_weight=w, **base))
    want = block.norm_backward(U.f64(h), dn=U.f64(dn), pre=U.f64(w), pre_eps=1e-6)
    U.near(dh, want["dh"], want["dh_mag"], 2 * NORM_ROUNDINGS, "dh")
    U.near(dpre, want["dpre"], want["dpre_mag"], 2 * NORM_ROUNDINGS + T, "dpre")
    y, dr, gate = r(T, H, dtype=BF16), r(T, H, dtype=BF16), r(T)
    got, dy, dgate = dr.clone(), torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(T, device="cuda")
    a = B.make_args(B.mega_moe_norm_backward_args, dr=got, dh=got, dy=dy, dgate=dgate, y=y, gate=gate,
                    gate_kind=B.MEGA_MOE_GATE_TOKEN, gate_type=B.MEGA_MOE_F32, **{**base, "residual_scale": -2.0})
    assert B.mega_moe_norm_workspace_bytes(a) == 0
    B.mega_moe_norm_backward(a, U.current_stream())
    want = block.norm_backward(U.f64(h), U.f64(dr), None, U.f64(y), U.f64(gate), "token", scale=-2.0)
    U.near(got, want["dh"], want["dh_mag"], NORM_ROUNDINGS, "dh in place")
    U.near(dy, want["dy"], want["dy_mag"], NORM_ROUNDINGS, "dy")
    U.near(dgate, want["dgate"], want["dgate_mag"], 2 * NORM_ROUNDINGS, "dgate")
    dpre.fill_(5.0)
    a = B.make_args(B.mega_moe_norm_backward_args, dpre_weight=dpre, pre_weight=w, **{**base, "num_tokens": 0})
    U.finish_norm_backward(a)
    assert not dpre.any()


# ---- router product ----------------------------------------------------------------

# tokens, hidden, experts, weight type, extra elements per row
LOGITS = [(1, 8, 1, BF16, 0), (1, 7168, 32, BF16, 0), (3, 40, 5, F32, 8), (16, 128, 16, F32, 0), (17, 136, 33, BF16, 0),
          (64, 512, 64, F32, 0), (65, 1000, 100, BF16, 16), (129, 2048, 257, F32, 0), (33, 512, 1024, BF16, 0),
          (300, 896, 256, BF16, 0), (515, 1152, 300, F32, 8), (1100, 256, 7, BF16, 0), (2050, 640, 72, F32, 0)]


def _logits_inputs(T, H, E, wt, extra):
    r = _gen(7 * T + H + E)
    x, _ = U.padded(T, H, BF16, extra)
    x.copy_(r(T, H))
    x[:, H // 3] *= 50.0
    return x, r(E, H, dtype=wt, scale=0.02), r


def _logits_fields(T, H, E, wt, x, w, extra):
    return dict(num_tokens=T, hidden=H, num_experts=E, weight_type=U.TYPE[wt], x=x, w=w, x_stride=H + extra)


# products that go through tiles in LDS: few, some and many experts, one part of K
# and several, workgroups in pairs, odd sizes
LOGITS_LARGE = [(9001, 1032, 29, BF16, 8), (5003, 1160, 17, F32, 0), (5003, 904, 50, BF16, 0), (3300, 904, 61, F32, 16),
                (2050, 520, 330, BF16, 0), (1030, 776, 260, F32, 8), (8200, 72, 330, BF16, 0), (257, 7168, 512, BF16, 0),
                (8200, 4104, 130, F32, 8), (9001, 1160, 29, BF16, 8), (5003, 1480, 17, F32, 0),
                (5003, 1096, 50, BF16, 0), (13000, 72, 330, BF16, 0)]


@pytest.mark.parametrize("T,H,E,wt,extra", LOGITS + LOGITS_LARGE)
def test_router_logits_match_the_reference(T, H, E, wt, extra):
    x, w, _ = _logits_inputs(T, H, E, wt, extra)
    logits, buf = U.padded(T, E, F32, extra)
    a = B.make_args(B.mega_moe_router_logits_args, logits=logits, logits_stride=E + extra,
                    **_logits_fields(T, H, E, wt, x, w, extra))
    B.set_args(a, **U.workspace(B.mega_moe_router_logits_workspace_bytes(a)))
    B.mega_moe_router_logits(a, U.current_stream())
    torch.cuda.synchronize()
    want, mag = block.router_logits(U.f64(x), U.f64(w))
    # products are exact; H adds (of three times as many terms with float32 weights)
    U.near(logits, want, mag, H + 16, "logits")
    if extra:
        assert torch.all(buf[:, E:] == 7.0)


# gradients of more than two workgroups to a compute unit
@pytest.mark.parametrize("T,H,E,wt,extra", LOGITS + [(8200, 1032, 66, F32, 8), (4100, 2056, 70, BF16, 0)])
@pytest.mark.parametrize("add", [False, True])
def test_router_logits_backward_matches_the_reference(T, H, E, wt, extra, add):
    x, w, r = _logits_inputs(T, H, E, wt, extra)
    d, _ = U.padded(T, E, F32, extra)
    d.copy_(r(T, E, scale=0.01))
    dx, dx_buf = U.padded(T, H, BF16, extra)
    before = r(T, H, dtype=BF16) if add else None
    dw = torch.full((E, H), 7.0, device="cuda")
    a = B.make_args(B.mega_moe_router_logits_args, dlogits=d, dlogits_stride=E + extra, dx=dx, dx_stride=H + extra,
                    dw=dw, dx_add=before, **_logits_fields(T, H, E, wt, x, w, extra))
    B.set_args(a, **U.workspace(B.mega_moe_router_logits_workspace_bytes(a)))
    B.mega_moe_router_logits_backward(a, U.current_stream())
    torch.cuda.synchronize()
    want = block.router_logits_backward(U.f64(d), U.f64(x), U.f64(w), U.f64(before))
    # dx: a float32 operand is held in two BF16 terms, so cut below 2^-16 of
    # itself (2^8 u), one or two operands; then E adds
    U.near(dx, want["dx"], want["dx_mag"], 2 * 2 ** 8 + E + 16, "dx")
    U.near(dw, want["dw"], want["dw_mag"], T + 16, "dw")
    if extra:
        assert torch.all(dx_buf[:, H:] == 7.0)


@pytest.mark.parametrize("T,H,E,wt", [(300, 264, 20, BF16), (70, 1032, 68, F32), (2100, 520, 64, BF16)])
def test_router_logits_backward_of_views_equals_that_of_copies(T, H, E, wt):
    # rows of dlogits that start between 16-byte words, and rows of a wider array
    # with NaN around them
    x, w, r = _logits_inputs(T, H, E, wt, 0)
    d = r(T, E, scale=0.01)
    out = []
    for lead, tail in ((0, 0), (1, 3), (4, 4), (2, 1)):
        wide = torch.full((T, lead + E + tail), float("nan"), device="cuda")
        wide[:, lead:lead + E] = d
        dx, dw = torch.empty(T, H, dtype=BF16, device="cuda"), torch.empty(E, H, device="cuda")
        a = B.make_args(B.mega_moe_router_logits_args, dlogits=wide[:, lead:], dlogits_stride=lead + E + tail, dx=dx,
                        dw=dw, **_logits_fields(T, H, E, wt, x, w, 0))
        B.set_args(a, **U.workspace(B.mega_moe_router_logits_workspace_bytes(a)))
        B.mega_moe_router_logits_backward(a, U.current_stream())
        out.append((dx, dw))
    torch.cuda.synchronize()
    want = block.router_logits_backward(U.f64(d), U.f64(x), U.f64(w))
    U.near(out[0][0], want["dx"], want["dx_mag"], 2 * 2 ** 8 + E + 16, "dx")
    U.near(out[0][1], want["dw"], want["dw_mag"], T + 16, "dw")
    for dx, dw in out[1:]:
        assert torch.equal(dx, out[0][0]) and torch.equal(dw, out[0][1])


def test_router_logits_backward_of_parts_and_no_tokens():
    T, H, E = 20, 64, 6
    x, w, r = _logits_inputs(T, H, E, F32, 0)
    d = r(T, E)
    for name in ("dx", "dw"):
        out = torch.empty(T, H, dtype=BF16, device="cuda") if name == "dx" else torch.empty(E, H, device="cuda")
        a = B.make_args(B.mega_moe_router_logits_args, dlogits=d, **{name: out}, **_logits_fields(T, H, E, F32, x, w, 0))
        B.set_args(a, **U.workspace(B.mega_moe_router_logits_workspace_bytes(a)))
        B.mega_moe_router_logits_backward(a, U.current_stream())
        want = block.router_logits_backward(U.f64(d), U.f64(x), U.f64(w))
        U.near(out, want[name], want[name + "_mag"], 2 * 2 ** 8 + T + E + 16, name)
    # in place: dx is dx_add
    dx = r(T, H, dtype=BF16)
    before = dx.clone()
    a = B.make_args(B.mega_moe_router_logits_args, dlogits=d, dx=dx, dx_add=dx, **_logits_fields(T, H, E, F32, x, w, 0))
    B.set_args(a, **U.workspace(B.mega_moe_router_logits_workspace_bytes(a)))
    B.mega_moe_router_logits_backward(a, U.current_stream())
    want = block.router_logits_backward(U.f64(d), U.f64(x), U.f64(w), U.f64(before))
    U.near(dx, want["dx"], want["dx_mag"], 2 * 2 ** 8 + E + 16, "dx in place")
    dw = torch.full((E, H), 5.0, device="cuda")
    a = B.make_args(B.mega_moe_router_logits_args, dw=dw, num_tokens=0, hidden=H, num_experts=E,
                    weight_type=B.MEGA_MOE_F32)
    B.set_args(a, **U.workspace(B.mega_moe_router_logits_workspace_bytes(a)))
    B.mega_moe_router_logits_backward(a, U.current_stream())
    assert not dw.any()


# ---- selection -------------------------------------------------------------------------

# tokens, experts, k, score, logits type, bias, groups, kept groups, group top, renormalize
TOPK = [
    (1, 1, 1, "softmax", F32, False, 1, 1, 1, True),
    (1, 8, 2, "softmax", F32, False, 1, 1, 1, True),
    (5, 32, 8, "softmax", BF16, False, 1, 1, 1, False),
    (130, 64, 6, "sigmoid", F32, True, 1, 1, 1, True),
    (33, 65, 65, "softmax", F32, True, 1, 1, 1, True),
    (9, 100, 7, "sigmoid", BF16, False, 1, 1, 1, False),
    (70, 128, 4, "softmax", F32, True, 4, 2, 1, True),
    (101, 256, 8, "sigmoid", F32, True, 8, 4, 2, True),
    (40, 160, 6, "softmax", BF16, False, 8, 3, 1, True),
    (12, 384, 12, "sigmoid", F32, False, 6, 1, 2, False),
    (6, 512, 100, "softmax", F32, False, 1, 1, 1, True),
    (3, 1024, 1024, "sigmoid", F32, True, 1, 1, 1, True),
    (4, 1000, 16, "softmax", BF16, True, 50, 7, 2, True),
    (3, 128, 64, "sigmoid", F32, True, 64, 32, 2, True),
]


def _topk(logits, k, score, bias=None, mask=None, groups=1, kept=1, top=1, renormalize=True, scale=2.5, stride=0):
    T, E = logits.shape
    idx = torch.full((T, k), 99, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), 7.0, device="cuda")
    a = B.make_args(B.mega_moe_router_topk_args, num_tokens=T, num_experts=E, num_topk=k,
                    logits_type=U.TYPE[logits.dtype], score=U.SCORE[score], renormalize=int(renormalize),
                    num_groups=groups, topk_groups=kept, group_top=top, weight_scale=scale, logits=logits, bias=bias,
                    token_mask=mask, topk_idx=idx, topk_weights=w, logits_stride=stride)
    B.mega_moe_router_topk(a, U.current_stream())
    torch.cuda.synchronize()
    return idx, w


def _check_topk(logits, k, score, bias=None, mask=None, groups=1, kept=1, top=1, renormalize=True, stride=0):
    idx, w = _topk(logits, k, score, bias, mask, groups, kept, top, renormalize, 2.5, stride)
    want_idx, want = block.router_topk(U.f64(logits), k, score, U.f64(bias), None if mask is None else mask.cpu().numpy(),
                                       renormalize, 2.5, groups, kept, top)
    assert np.array_equal(idx.cpu().numpy(), want_idx)
    # exp and the division carry a few roundings, l - max half of one of |l| <= 8,
    # and the sums E / 64 + 6 and k adds
    U.near(w, want, want, 32 + logits.shape[1] // 64 + k, "topk_weights")


# batches above 2048 tokens give a token fewer lanes
TOPK_LARGE = [
    (2100, 100, 6, "softmax", F32, False, 1, 1, 1, True),
    (2060, 256, 8, "sigmoid", F32, True, 8, 4, 2, True),
    (2050, 96, 4, "softmax", BF16, True, 12, 5, 1, False),
    (2049, 300, 31, "sigmoid", F32, True, 1, 1, 1, True),
    (2052, 200, 30, "sigmoid", F32, True, 5, 2, 2, True),
    (4100, 128, 8, "softmax", F32, False, 1, 1, 1, True),
    (4098, 112, 6, "sigmoid", BF16, True, 7, 3, 2, True),
]


@pytest.mark.parametrize("T,E,k,score,lt,bias,groups,kept,top,renormalize", TOPK + TOPK_LARGE)
def test_selection_matches_the_reference(T, E, k, score, lt, bias, groups, kept, top, renormalize):
    r = _gen(T + 3 * E + k)
    logits = r(T, E, dtype=lt)
    b = r(E, scale=0.05) if bias else None
    mask = torch.from_numpy((np.arange(T) % 5 != 3).astype(np.uint8)).cuda()
    _check_topk(logits, k, score, b, None, groups, kept, top, renormalize)
    _check_topk(logits, k, score, b, mask, groups, kept, top, renormalize)
    wide, _ = U.padded(T, E, lt, 5)
    wide.copy_(logits)
    _check_topk(wide, k, score, b, mask, groups, kept, top, renormalize, stride=E + 5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("biased", [False, True])
def test_selection_of_masked_experts_ties_and_nan(score, groups, biased):
    T, E, k = 12, 48, 5
    r = _gen(9)
    logits = torch.round(r(T, E) * 2) / 2            # many exact ties
    logits[1, 3:] = -float("inf")                    # fewer experts than slots
    logits[2] = -float("inf")                        # none at all
    logits[3, ::2] = -float("inf")
    logits[4, :13] = -float("inf")                   # a whole group and one more
    bias = None
    if biased:
        bias = torch.zeros(E, device="cuda")
        bias[7] = -float("inf")                      # an expert taken out by its bias
    _check_topk(logits, k, score, bias, None, groups, 2, 2)
    # NaN: never taken; the softmax's sum is NaN, a sigmoid's neighbours are not
    logits[5, 11] = float("nan")
    idx, w = _topk(logits[5:6].contiguous(), k, score, None, None, 1, 1, 1)
    assert 11 not in idx.tolist()[0]
    assert torch.isnan(w).all() == (score == "softmax")


def test_selection_follows_near_ties_exactly():
    # neighbouring float32 logits, and biased scores that differ in the 12th digit
    logits = torch.full((1, 64), 0.5, device="cuda")
    step = np.nextafter(np.float32(0.5), np.float32(1.0))
    logits[0, 40] = float(step)
    assert _topk(logits, 2, "softmax")[0].tolist() == [[40, 0]]
    a = np.float32(0.3)
    logits = torch.tensor([[float(a), float(np.nextafter(a, np.float32(1))), 0.0, 0.0]], device="cuda")
    s = 1.0 / (1.0 + np.exp(-np.float64(logits[0].cpu().numpy())))
    bias = torch.zeros(4, device="cuda")
    bias[0] = float(np.float32(s[1] - s[0]) * np.float32(0.999))
    assert _topk(logits, 1, "sigmoid", bias)[0].tolist() == [[1]]
    bias[0] = float(np.float32(s[1] - s[0]) * np.float32(1.001))
    assert _topk(logits, 1, "sigmoid", bias)[0].tolist() == [[0]]


# few and many slots (the keys of a lane in order or not), and group sizes of one
# and several times 16, with scores that tie within a lane and across lanes
@pytest.mark.parametrize("T,E,groups,ks", [(40, 64, 4, (1, 2, 3, 9)), (2100, 64, 1, (1, 9)), (2100, 256, 16, (4, 5, 11)),
                                           (60, 240, 5, (1, 2, 3, 29)), (2060, 192, 4, (2, 8, 27)),
                                           (50, 512, 8, (1, 4, 5, 40)), (30, 1024, 64, (8, 9, 61)),
                                           (30, 960, 4, (2, 8, 13))])
def test_selection_of_few_and_many_slots_among_ties(T, E, groups, ks):
    r = _gen(T + E)
    logits = torch.round(r(T, E) * 4) / 4            # about 30 values
    logits[::7, : E // groups] = -float("inf")
    bias = torch.round(r(E) * 2) / 2
    for k in ks:
        _check_topk(logits, k, "softmax")
        _check_topk(logits, k, "sigmoid", bias)
        if groups > 1:
            need = -(-k * groups // E)                   # groups that hold k experts
            _check_topk(logits, k, "sigmoid", bias, None, groups, max(need, 2), 2)
            _check_topk(logits, k, "sigmoid", bias, None, groups, need, 1)


@pytest.mark.parametrize("T,E", [(300, 64), (300, 256), (2100, 128), (200, 512)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [1, 4])
def test_selection_orders_near_ties_in_float64(T, E, score, groups):
    # every row: a few values, copied over the experts, some moved by one step of
    # float32: groups and experts that float32 scores cannot tell apart
    rng = np.random.default_rng(T + E + groups)
    base = rng.standard_normal((T, 4)).astype(np.float32)
    l = np.take_along_axis(base, rng.integers(0, 4, (T, E)), axis=1)
    moved = rng.random((T, E)) < 0.3
    l = np.where(moved, np.nextafter(l, np.where(rng.random((T, E)) < 0.5, np.inf, -np.inf).astype(np.float32)), l)
    bias = np.where(rng.random(E) < 0.2, np.float32(2.0 ** -24), np.float32(0.0)).astype(np.float32)
    k, kept, top = 7, 2, 2
    logits, b = torch.from_numpy(l).cuda(), torch.from_numpy(bias).cuda()
    idx, _ = _topk(logits, k, score, b, None, groups, kept, top)
    want, _ = block.router_topk(l, k, score, bias, None, True, 2.5, groups, kept, top)
    undecided = _beyond_float64(l, k, score, bias, groups, kept, top)
    assert undecided.mean() < 0.2
    same = np.all(idx.cpu().numpy() == want, axis=1)
    assert np.all(same | undecided), np.argwhere(~(same | undecided))[:5].tolist()


def _beyond_float64(l, k, score, bias, groups, kept, top):
    """Rows whose order float64 cannot tell.  A key there is exp (one step), a
    division and a sum: under four half steps of 1 (2^-53 each) from the true
    one, and a group's score, the sum of two, under ten.  Two float64
    computations of the same row may thus differ in the order of neighbours
    nearer than twice that; 2^-48 is above it.  Equal logits with equal biases
    are no such case: they give equal keys in both, and groups of equal pairs
    equal scores.  Judged in 64-bit mantissas (2^-64)."""
    x = l.astype(np.longdouble)
    s = np.exp(x - x.max(axis=1, keepdims=True))
    s = s / s.sum(axis=1, keepdims=True) if score == "softmax" else 1 / (1 + np.exp(-x))
    out = np.zeros(len(l), bool)
    size = l.shape[1] // groups
    near = np.longdouble(2.0 ** -48)
    for t in range(len(l)):
        c = s[t] + bias.astype(np.longdouble)
        what = [(l[t, e], bias[e]) for e in range(l.shape[1])]
        live = list(range(l.shape[1]))
        if groups > 1:
            best = [sorted(range(g * size, (g + 1) * size), key=lambda e: -c[e])[:top] for g in range(groups)]
            order = sorted(range(groups), key=lambda g: (-sum(c[e] for e in best[g]), g))
            for a in order[:kept]:
                for z in order[kept:]:
                    if sorted(what[e] for e in best[a]) != sorted(what[e] for e in best[z]):
                        out[t] |= sum(c[e] for e in best[a]) - sum(c[e] for e in best[z]) < near
            live = [e for e in live if e // size in order[:kept]]
        order = sorted(live, key=lambda e: (-c[e], e))[:k + 1]
        for a, z in zip(order, order[1:]):
            out[t] |= what[a] != what[z] and c[a] - c[z] < near
    return out


# ---- losses and gradients ------------------------------------------------------------------

# tokens, experts, k, score, logits type, cuts (None: one sequence), masked tokens
SEQ = [
    (1, 4, 1, "softmax", F32, None, False),
    (1, 1, 1, "sigmoid", F32, [0, 1], False),
    (50, 32, 8, "softmax", F32, None, True),
    (50, 32, 8, "sigmoid", BF16, [0, 1, 1, 20, 41], False),
    (333, 100, 3, "softmax", BF16, [5, 5, 6, 130, 300], True),
    (700, 256, 8, "sigmoid", F32, [0, 333, 700], True),
    (129, 300, 2, "softmax", F32, [0, 64, 128, 129], False),
    (40, 1024, 4, "sigmoid", F32, [0, 40], True),
    (64, 8, 70, "softmax", F32, [0, 0, 0], False),
    (3000, 16, 2, "softmax", F32, None, False),
    (2100, 200, 4, "softmax", F32, [3, 700, 2050], True),
    (2100, 70, 6, "sigmoid", BF16, list(range(0, 2101, 21)), False),
    (4100, 120, 5, "softmax", F32, [0, 9, 4000], True),
]


def _route(T, E, k, score, lt, cuts, masked):
    r = _gen(T + E + k)
    logits = r(T, E, dtype=lt)
    idx = torch.randint(0, E, (T, k), generator=torch.Generator().manual_seed(T), dtype=torch.int32)
    idx[::7, 0] = -1                       # empty slots, and indices that no expert has
    idx[1::9, k - 1] = E
    mask = (torch.arange(T) % 6 != 5).to(torch.uint8).cuda() if masked else None
    cu = None if cuts is None else torch.tensor(cuts, dtype=torch.int32).cuda()
    return logits, idx.cuda(), mask, cu, r


def _balance(logits, idx, score, mask, cu, stride=0):
    T, E = logits.shape
    k = idx.shape[1]
    B_ = 1 if cu is None else cu.numel() - 1
    o = dict(loss=torch.full((2,), 7.0, device="cuda"), counts=torch.full((B_, E), 7, dtype=torch.int32, device="cuda"),
             tokens=torch.full((B_ + 2,), 7, dtype=torch.int32, device="cuda"), probs=torch.full((B_, E), 7.0, device="cuda"))
    a = B.make_args(B.mega_moe_balance_loss_args, num_tokens=T, num_experts=E, num_topk=k,
                    logits_type=U.TYPE[logits.dtype], score=U.SCORE[score], num_sequences=0 if cu is None else B_,
                    balance_coeff=0.5, z_coeff=0.25, logits=logits, topk_idx=idx, token_mask=mask, cu_seqlens=cu,
                    logits_stride=stride, **o)
    B.set_args(a, **U.workspace(B.mega_moe_balance_loss_workspace_bytes(a)))
    B.mega_moe_balance_loss(a, U.current_stream())
    torch.cuda.synchronize()
    return o


def _np(t):
    return None if t is None else t.cpu().numpy()


@pytest.mark.parametrize("T,E,k,score,lt,cuts,masked", SEQ)
def test_balance_loss_matches_the_reference(T, E, k, score, lt, cuts, masked):
    logits, idx, mask, cu, _ = _route(T, E, k, score, lt, cuts, masked)
    o = _balance(logits, idx, score, mask, cu)
    want = block.balance_loss(U.f64(logits), _np(idx), score, cuts, _np(mask), 0.5, 0.25)
    assert np.array_equal(_np(o["counts"]), want["counts"])
    assert np.array_equal(_np(o["tokens"]), want["tokens"])
    # p: 32 roundings and E / 64 + 6 adds; then at most T adds of positive terms,
    # E of them in the loss, and one per sequence
    adds = 32 + E // 64 + T
    U.near(o["probs"], want["probs"], want["probs"], adds, "probs")
    U.near(o["loss"], want["loss"], want["loss_mag"], adds + E + len(cuts or []), "loss")


def test_balance_loss_without_tokens_and_with_an_empty_row():
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    o = _balance(torch.zeros(0, 5, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda"), "softmax", None, cu)
    assert not o["loss"].any() and not o["counts"].any() and not o["tokens"].any() and not o["probs"].any()
    logits = torch.zeros(2, 4, device="cuda")
    logits[0] = -float("inf")
    idx = torch.tensor([[-1], [2]], dtype=torch.int32, device="cuda")
    o = _balance(logits, idx, "softmax", None, None)
    want = block.balance_loss(U.f64(logits), _np(idx), "softmax", None, None, 0.5, 0.25)
    assert np.allclose(_np(o["loss"]), want["loss"], rtol=1e-6) and np.array_equal(_np(o["tokens"]), [2, 2, 1])


@pytest.mark.parametrize("T,E,k,score,lt,cuts,masked", SEQ)
@pytest.mark.parametrize("parts", ["weights", "losses", "both"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_router_backward_matches_the_reference(T, E, k, score, lt, cuts, masked, parts, renormalize):
    logits, idx, mask, cu, r = _route(T, E, k, score, lt, cuts, masked)
    B_ = 1 if cu is None else len(cuts) - 1
    dw, dloss = r(T, k), r(2)
    ref = block.balance_loss(U.f64(logits), _np(idx), score, cuts, _np(mask), 0.5, 0.25)
    counts = torch.from_numpy(ref["counts"].astype(np.int32)).cuda()
    tokens = torch.from_numpy(ref["tokens"].astype(np.int32)).cuda()
    d, buf = U.padded(T, E, F32, 3)
    f = dict(num_tokens=T, num_experts=E, num_topk=k, logits_type=U.TYPE[lt], score=U.SCORE[score], logits=logits,
             token_mask=mask, dlogits=d, dlogits_stride=E + 3)
    want = dict(mask=_np(mask))
    if parts != "losses":
        f.update(topk_idx=idx, dweights=dw, renormalize=int(renormalize), weight_scale=1.5)
        want.update(idx=_np(idx), dweights=U.f64(dw), renormalize=renormalize, scale=1.5)
    if parts != "weights":
        f.update(dloss=dloss, cu_seqlens=cu, num_sequences=0 if cu is None else B_, counts=counts, tokens=tokens,
                 balance_coeff=0.5, z_coeff=0.25)
        want.update(dloss=U.f64(dloss), cu=cuts, counts=ref["counts"], tokens=ref["tokens"], k=k, balance_coeff=0.5,
                    z_coeff=0.25)
    B.mega_moe_router_backward(B.make_args(B.mega_moe_router_backward_args, **f), U.current_stream())
    torch.cuda.synchronize()
    g, mag = block.router_backward(U.f64(logits), score, **want)
    # scores: 32 roundings and E / 64 + 6 adds; the sums over slots k, over experts the same again
    U.near(d, g, mag, 2 * (48 + E // 64) + 2 * k, "dlogits")
    assert torch.all(buf[:, E:] == 7.0)


def test_router_backward_of_a_repeated_expert_and_an_empty_row():
    T, E, k = 3, 6, 3
    r = _gen(21)
    logits = r(T, E)
    logits[1] = -float("inf")
    logits[2, 3:] = -float("inf")
    idx = torch.tensor([[2, 2, 4], [-1, -1, -1], [0, 1, -1]], dtype=torch.int32, device="cuda")
    dw = r(T, k)
    for score in ("softmax", "sigmoid"):
        for renormalize in (0, 1):
            o = _balance(logits, idx, score, None, None)
            d = torch.full((T, E), 7.0, device="cuda")
            dloss = torch.ones(2, device="cuda")
            B.mega_moe_router_backward(
                B.make_args(B.mega_moe_router_backward_args, num_tokens=T, num_experts=E, num_topk=k,
                            logits_type=B.MEGA_MOE_F32, score=U.SCORE[score], renormalize=renormalize, logits=logits,
                            topk_idx=idx, dweights=dw, dloss=dloss, counts=o["counts"], tokens=o["tokens"],
                            balance_coeff=0.5, z_coeff=0.25, dlogits=d), U.current_stream())
            g, mag = block.router_backward(U.f64(logits), score, _np(idx), U.f64(dw), bool(renormalize), 1.0, None,
                                           np.ones(2), None, _np(o["counts"]), _np(o["tokens"]), k, 0.5, 0.25)
            U.near(d, g, mag, 128, f"{score} {renormalize}")
            assert not d[1].any()


# ---- rows far apart: offsets beyond 32 bits -----------------------------------------------------

def test_offsets_beyond_32_bits():
    far = 1 << 31                        # elements from row to row: rows 0, 4 GiB and 8 GiB apart in BF16
    r = _gen(31)
    buf = torch.empty(2 * far + 4096, dtype=BF16, device="cuda")
    T, H = 3, 256
    h = buf.as_strided((T, H), (far, 1))
    h.copy_(r(T, H))
    w, n = r(H), torch.empty(T, H, dtype=BF16, device="cuda")
    B.mega_moe_norm(B.make_args(B.mega_moe_norm_args, num_tokens=T, hidden=H, weight_type=B.MEGA_MOE_F32, pre_eps=1e-6,
                                residual_scale=1.0, h=h, h_stride=far, r=h, r_stride=far, n=n, pre_weight=w),
                    U.current_stream())
    want = block.norm(U.f64(h), pre=U.f64(w), pre_eps=1e-6)
    U.near(n, want["n"], want["n_mag"], NORM_ROUNDINGS, "n")
    dh, dpre = buf.as_strided((T, H), (far, 1), 1024), torch.empty(H, device="cuda")
    dn = r(T, H, dtype=BF16)
    U.finish_norm_backward(B.make_args(
        B.mega_moe_norm_backward_args, num_tokens=T, hidden=H, weight_type=B.MEGA_MOE_F32, pre_eps=1e-6, residual_scale=1.0,
        r=h, r_stride=far, dn=dn, pre_weight=w, dh=dh, dh_stride=far, dpre_weight=dpre))
    want = block.norm_backward(U.f64(h), dn=U.f64(dn), pre=U.f64(w), pre_eps=1e-6)
    U.near(dh, want["dh"], want["dh_mag"], 2 * NORM_ROUNDINGS, "dh")
    E, k = 40, 4
    l = buf.as_strided((T, E), (far, 1), 2048)
    l.copy_(r(T, E))
    _check_topk(l, k, "softmax", stride=far)
    idx, _ = block.router_topk(U.f64(l), k, "softmax")
    o = _balance(l, torch.from_numpy(idx).cuda(), "softmax", None, None, stride=far)
    want = block.balance_loss(U.f64(l), idx, "softmax", None, None, 0.5, 0.25)
    U.near(o["loss"], want["loss"], want["loss_mag"], 128, "loss")
    del buf, h, dh, l
    # the router's product: rows 2^22 elements apart, beyond 2^32 at row 1024
    T, H, E, far = 1030, 64, 8, 1 << 22
    buf = torch.empty((T - 1) * far + H, dtype=BF16, device="cuda")
    x, w, d = buf.as_strided((T, H), (far, 1)), r(E, H), r(T, E)
    x.copy_(r(T, H))
    logits, dw = torch.empty(T, E, device="cuda"), torch.empty(E, H, device="cuda")
    a = B.make_args(B.mega_moe_router_logits_args, num_tokens=T, hidden=H, num_experts=E, weight_type=B.MEGA_MOE_F32, x=x,
                    x_stride=far, w=w, logits=logits, dlogits=d, dw=dw)
    B.set_args(a, **U.workspace(B.mega_moe_router_logits_workspace_bytes(a)))
    B.mega_moe_router_logits(a, U.current_stream())
    B.mega_moe_router_logits_backward(a, U.current_stream())
    xs = U.f64(x)
    want, mag = block.router_logits(xs, U.f64(w))
    U.near(logits, want, mag, H + 16, "logits")
    want = block.router_logits_backward(U.f64(d), xs, U.f64(w))
    U.near(dw, want["dw"], want["dw_mag"], T + 16, "dw")
