"""The dense path's operators over sizes, types, layouts, strides and special
values against float64, with tolerances counted in roundings."""

import numpy as np
import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from oracle import dense
from tests import block_util as U
from tests import dense_util as D

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


# ---- products ------------------------------------------------------------------

SIZES = [(1, 128, 8), (1, 7168, 264), (2, 256, 128), (7, 1280, 1000), (16, 512, 136), (17, 384, 4096), (32, 2048, 64), (33, 128, 72),
         (64, 1024, 520), (65, 256, 128), (127, 896, 256), (128, 2048, 7168), (130, 4096, 264), (257, 640, 512), (300, 128, 1032),
         (1000, 1152, 904), (4096, 128, 4096), (2049, 384, 2056)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("out_type", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("scale", ["block", "row"])
def test_product(m, k, n, out_type, scale):
    g = D.generator(m * 7 + n)
    a, a_sf = D.operand(g, m, k)
    b, b_sf = D.operand(g, n, k, scale)
    add = D.randn(g, m, n, scale=30.0, dtype=out_type) if (m + n) % 16 else None
    out = torch.full((m, n), 7.0, dtype=out_type, device="cuda")
    D.product(a, a_sf, b, b_sf, out, scale, add)
    D.check_product(out, a, a_sf, b, b_sf, scale, add)


# sizes that go through each of the kinds of tiles, whole and split, with rows and columns left over
KINDS = [(33, 1664, 8440), (33, 10240, 1112), (133, 640, 11064), (1027, 10240, 72), (1025, 10240, 8), (1, 1152, 8200), (1, 16384, 520),
         (129, 10240, 5576), (65, 2944, 8424), (67, 7168, 2744), (259, 128, 10952), (65, 128, 8840), (1025, 128, 7208), (33, 896, 4136),
         (1, 1664, 12408), (65, 16384, 1416), (1, 10240, 136), (13, 384, 6504), (3, 16384, 1032), (523, 16384, 8)]


@pytest.mark.parametrize("m,k,n", KINDS)
@pytest.mark.parametrize("scale", ["block", "row"])
def test_product_by_every_tile(m, k, n, scale):
    g = D.generator(m + n)
    a, a_sf = D.operand(g, m, k)
    b, b_sf = D.operand(g, n, k, scale)
    ref = D.reference(a, a_sf, b, b_sf, scale)
    for out_type in (BF16, F32):
        out = torch.full((m + 1, n), 7.0, dtype=out_type, device="cuda")
        D.product(a, a_sf, b, b_sf, out[:m], scale)
        D.check_product(out[:m], a, a_sf, b, b_sf, scale, ref=ref)
        assert bool((out[m] == 7).all())


@pytest.mark.parametrize("m,k,n", [(5, 256, 72), (70, 1024, 136), (300, 512, 264), (4100, 128, 4104)])
@pytest.mark.parametrize("out_type", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("scale", ["block", "row"])
def test_product_of_spaced_rows_leaves_the_gaps(m, k, n, out_type, scale):
    g = D.generator(m)
    a, a_sf = D.operand(g, m, k)
    b, b_sf = D.operand(g, n, k, scale)
    add = D.randn(g, m, n, dtype=out_type)
    av, _ = D.spaced(a, 48, 0x7F)                # NaN codes and scales behind every row
    bv, _ = D.spaced(b, 16, 0x7F)
    asv, _ = D.spaced(a_sf, 3, float("nan"))
    bsv, _ = D.spaced(b_sf, 1, float("nan"))
    addv, _ = D.spaced(add, 24, float("nan"))
    out, buf = U.padded(m, n, out_type, 40)
    D.product(av, asv, bv, bsv, out, scale, addv, a_stride=k + 48, b_stride=k + 16, a_sf_stride=k // 128 + 3,
              b_sf_stride=k // 128 + 1, add_stride=n + 24, out_stride=n + 40)
    D.check_product(out, a, a_sf, b, b_sf, scale, add)
    assert bool((buf[:, n:] == 7.0).all())


@pytest.mark.parametrize("m,k,n", [(3, 512, 64), (200, 4096, 128), (4096, 128, 4096)])
@pytest.mark.parametrize("out_type", [BF16, F32], ids=["bf16", "f32"])
def test_product_adds_to_its_own_output(m, k, n, out_type):
    g = D.generator(3)
    a, a_sf = D.operand(g, m, k)
    b, b_sf = D.operand(g, n, k, "row")
    out = D.randn(g, m, n, scale=5.0, dtype=out_type)
    before = out.clone()
    D.product(a, a_sf, b, b_sf, out, "row", out)
    D.check_product(out, a, a_sf, b, b_sf, "row", before)


@pytest.mark.parametrize("m,n", [(1, 64), (150, 136)])
@pytest.mark.parametrize("add", [False, True])
def test_product_without_columns_is_what_is_added(m, n, add):
    old = D.randn(D.generator(1), m, n, dtype=BF16) if add else None
    out = torch.full((m, n), 7.0, dtype=BF16, device="cuda")
    args = B.make_args(B.mega_moe_product_args, m=m, n=n, k=0, out_type=B.MEGA_MOE_BF16, add=old, out=out)
    B.mega_moe_product(args, U.current_stream())
    assert torch.equal(out, old if add else torch.zeros_like(out))


@pytest.mark.parametrize("m,k,n", [(1, 7168, 64), (40, 4096, 72), (130, 2048, 264), (520, 1024, 256)])
@pytest.mark.parametrize("scale", ["block", "row"])
def test_float32_products_of_small_integers_are_exact(m, k, n, scale):
    g = D.generator(m + k)
    values = torch.tensor([0.0, 1.0, -1.0, 2.0, -3.0, 0.5, -0.5, 1.5], device="cuda")

    def codes(rows):
        v = values[torch.randint(0, len(values), (rows, k), generator=g, device="cuda")]
        return v.to(torch.float8_e4m3fn).view(torch.uint8), v.double().cpu()

    (a, av), (b, bv) = codes(m), codes(n)
    a_sf = torch.exp2(torch.randint(-3, 3, (m, k // 128), generator=g, device="cuda").float())
    b_sf = torch.exp2(torch.randint(-2, 2, (n if scale == "row" else D.up128(n) // 128, k // 128), generator=g, device="cuda").float())
    out = torch.empty(m, n, device="cuda")
    D.product(a, a_sf, b, b_sf, out, scale)
    wa, wb = dense.wide_scales(U.f64(a_sf), m, True), dense.wide_scales(U.f64(b_sf), n, scale == "row")
    # sums of multiples of 2^-7 below 2^17: exact in any order
    assert np.array_equal(U.f64(out), (av.numpy() * wa) @ (bv.numpy() * wb).T)


@pytest.mark.parametrize("out_type", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("m,n", [(4, 64), (100, 200), (2200, 8192)])
def test_nan_infinity_and_zero_scales_stay_in_their_rows(m, n, out_type):
    g = D.generator(9)
    k = 384
    a, a_sf = D.operand(g, m, k)
    b, b_sf = D.operand(g, n, k, "row")
    a_sf[0, 1] = 0.0
    b_sf[0, :] = 0.0
    clean = torch.empty(m, n, dtype=out_type, device="cuda")
    D.product(a, a_sf, b, b_sf, clean, "row")
    D.check_product(clean, a, a_sf, b, b_sf, "row")
    assert bool((clean[:, 0] == 0).all())
    a2, a_sf2, b2 = a.clone(), a_sf.clone(), b.clone()
    a2[1, 5] = 0x7F
    b2[n - 1, 300] = 0xFF
    a_sf2[2, 2] = float("inf")
    out = torch.empty_like(clean)
    D.product(a2, a_sf2, b2, b_sf, out, "row")
    assert bool(out[1].isnan().all()) and bool(out[:, n - 1].isnan().all())
    assert not bool(out[2].isfinite().any())
    rest = [i for i in range(m) if i not in (1, 2)]
    assert torch.equal(out[rest, :n - 1], clean[rest, :n - 1])


def test_product_beyond_32_bit_offsets():
    g = D.generator(4)
    m, k, n, stride = 1100, 256, 136, 1 << 22
    a, a_sf = D.operand(g, m, k)
    b, b_sf = D.operand(g, n, k, "block")
    big = torch.empty((m - 1) * stride + k, dtype=torch.uint8, device="cuda")
    far = big.as_strided((m, k), (stride, 1))
    far.copy_(a)
    for out_type in (BF16, F32):
        out = torch.empty(m, n, dtype=out_type, device="cuda")
        D.product(far, a_sf, b, b_sf, out, "block", a_stride=stride)
        D.check_product(out, a, a_sf, b, b_sf, "block")
    out_stride = 1 << 21
    wide = torch.empty((m - 1) * out_stride + n, dtype=BF16, device="cuda").as_strided((m, n), (out_stride, 1))
    D.product(a, a_sf, b, b_sf, wide, "block", out_stride=out_stride)
    D.check_product(wide, a, a_sf, b, b_sf, "block")


def test_same_call_gives_the_same_bits():
    g = D.generator(8)
    for m, k, n in ((1, 7168, 4096), (128, 2048, 7168), (513, 4096, 1024)):
        a, a_sf = D.operand(g, m, k)
        b, b_sf = D.operand(g, n, k, "block")
        outs = [torch.empty(m, n, device="cuda", dtype=t) for t in (BF16, F32) for _ in range(3)]
        for o in outs:
            D.product(a, a_sf, b, b_sf, o, "block")
        assert all(torch.equal(o, outs[0]) for o in outs[1:3]) and all(torch.equal(o, outs[3]) for o in outs[4:])


# ---- operands --------------------------------------------------------------------

# silu: exp (2 roundings of its argument's magnitude are far below the others), sum, quotient, product
SWIGLU_ROUNDINGS = 12


def _quantize(x, up=None, scale="row", clamp=0.0, h=True, q=True, qt=True, **more):
    T, C = x.shape
    Tp, block = D.up128(T), scale == "block"
    new = lambda *s, dtype: torch.full(s, 0x55 if dtype == torch.uint8 else 7.0, dtype=dtype, device="cuda")   # noqa: E731
    o = dict(h=new(T, C, dtype=BF16) if h else None, q=new(T, C, dtype=torch.uint8) if q else None,
             q_sf=new(Tp // 128 if block else T, C // 128, dtype=F32) if q else None,
             qt=new(C, Tp, dtype=torch.uint8) if qt else None,
             qt_sf=new(C // 128 if block else C, Tp // 128, dtype=F32) if qt else None)
    f = dict(num_tokens=T, columns=C, x_type=U.TYPE[x.dtype], scale=D.SCALE[scale], activation_clamp=clamp, x=x, up=up,
             activation=B.MEGA_MOE_ACT_NONE if up is None else B.MEGA_MOE_ACT_SWIGLU, x_stride=x.stride(0),
             up_stride=0 if up is None else up.stride(0), **o)
    f.update(more)
    B.mega_moe_quantize(B.make_args(B.mega_moe_quantize_args, **f), U.current_stream())
    return o


def _check_quantize(o, v, scale, roundings, label=""):
    if o["h"] is not None:
        U.near(o["h"], v, np.abs(v), roundings, label + "h")
    if scale == "block":
        want = dense.block_quotients(v)
        if o["q"] is not None:
            D.check_codes(o["q"], o["q_sf"], want, roundings, label + "q")
        if o["qt"] is not None:
            wt = {"sf": want["sf"].T, "q": dense._padded(want["q"]).T}
            D.check_codes(o["qt"], o["qt_sf"], wt, roundings, label + "qt")
            if o["q"] is not None:       # the same codes, turned
                assert torch.equal(o["qt"][:, :v.shape[0]].t(), o["q"]) and torch.equal(o["qt_sf"].t(), o["q_sf"])
    else:
        if o["q"] is not None:
            D.check_codes(o["q"], o["q_sf"], dense.rows_quotients(v), roundings, label + "q")
        if o["qt"] is not None:
            D.check_codes(o["qt"], o["qt_sf"], dense.transposed_quotients(v), roundings, label + "qt")
    if o["qt"] is not None:
        assert bool((o["qt"][:, v.shape[0]:] == 0).all())


@pytest.mark.parametrize("T,C", [(1, 128), (3, 2048), (127, 256), (128, 384), (129, 128), (577, 512), (1000, 1152)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("scale", ["row", "block"])
@pytest.mark.parametrize("swiglu", [False, True])
def test_quantize(T, C, dtype, scale, swiglu):
    g = D.generator(T + C)
    both = D.randn(g, T, 2 * C, scale=2.0, dtype=dtype)
    both[0, :128] = 0.0                          # a block of zeros
    x, up = (both[:, :C], both[:, C:]) if swiglu else (both[:, :C], None)
    v = dense.swiglu(U.f64(x), U.f64(up)) if swiglu else U.f64(x)
    roundings = SWIGLU_ROUNDINGS if swiglu else 0
    full = _quantize(x, up, scale)
    _check_quantize(full, v, scale, roundings)
    # each output alone is the same
    for only in ("h", "q", "qt"):
        o = _quantize(x, up, scale, h=only == "h", q=only == "q", qt=only == "qt")
        for name, t in o.items():
            assert t is None or torch.equal(t, full[name]), (only, name)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_quantize_clamps_as_the_layer(dtype):
    g = D.generator(5)
    x, up = D.randn(g, 130, 256, scale=6.0, dtype=dtype), D.randn(g, 130, 256, scale=6.0, dtype=dtype)
    o = _quantize(x, up, clamp=4.0)
    _check_quantize(o, dense.swiglu(U.f64(x), U.f64(up), 4.0), "row", SWIGLU_ROUNDINGS)


@pytest.mark.parametrize("scale", ["row", "block"])
def test_quantize_at_the_ends_of_the_range(scale):
    x = torch.zeros(200, 256, device="cuda")
    x[0, :128] = torch.linspace(1e-44, 1e-38, 128, device="cuda")      # subnormal block
    x[1, 128:] = torch.linspace(-3e38, 3e38, 128, device="cuda")
    x[150, 7] = 448.0
    x[151, 7] = -1.0
    o = _quantize(x, None, scale, h=False)
    for q, sf, rows in ((o["q"], o["q_sf"], x.double()), (o["qt"], o["qt_sf"], torch.nn.functional.pad(x.double().t(), (0, 56)))):
        wide = sf.double()
        if scale == "block":
            wide = wide.repeat_interleave(128, dim=0)[:rows.shape[0]]
        wide = wide.repeat_interleave(128, dim=1)
        back = q.view(torch.float8_e4m3fn).double() * wide
        # float32's linspace runs over its largest value: row 1 holds infinities and NaN, and blocks with
        # them have no finite scale
        finite = wide.isfinite()
        assert bool(finite.any()) and not bool(finite.all())
        # half a step of the code, half the smallest step, and the scale's own rounding (a subnormal one loses up to 2^-150)
        near = (back - rows).abs() <= rows.abs() * (2.0 ** -4 + 2.0 ** -20) + wide * 2.0 ** -10 + 449 * 2.0 ** -150
        assert bool(near[finite].all())


def test_quantize_of_the_largest_values():
    x = torch.linspace(-1.0, 1.0, 256, device="cuda").repeat(3, 1) * torch.tensor([[3.4e38], [1e38], [1.2e-38]], device="cuda")
    o = _quantize(x, None, h=False, qt=False)
    back = o["q"].view(torch.float8_e4m3fn).double() * o["q_sf"].double().repeat_interleave(128, dim=1)
    wide = o["q_sf"].double().repeat_interleave(128, dim=1)
    assert bool(((back - x.double()).abs() <= x.double().abs() * (2.0 ** -4 + 2.0 ** -20) + wide * 2.0 ** -10 + 449 * 2.0 ** -150).all())


@pytest.mark.parametrize("scale", ["row", "block"])
def test_quantize_keeps_nan_in_its_block(scale):
    g = D.generator(6)
    x = D.randn(g, 300, 384, dtype=BF16)
    clean = _quantize(x, None, scale)
    x[130, 200] = float("nan")
    o = _quantize(x, None, scale)
    is_nan = lambda q: (q & 0x7F) == 0x7F        # noqa: E731
    if scale == "block":
        assert bool(is_nan(o["q"][128:256, 128:256]).all()) and bool(o["q_sf"][1, 1].isnan())
        keep = torch.ones(300, 384, dtype=torch.bool, device="cuda")
        keep[128:256, 128:256] = False
    else:
        assert bool(is_nan(o["q"][130, 128:256]).all()) and bool(o["q_sf"][130, 1].isnan())
        assert bool(is_nan(o["qt"][200, 128:256]).all()) and bool(o["qt_sf"][200, 1].isnan())
        keep = torch.ones(300, 384, dtype=torch.bool, device="cuda")
        keep[130, 128:256] = False
    assert torch.equal(o["q"][keep], clean["q"][keep])
    assert int(is_nan(o["q"]).sum()) == int((~keep).sum())


def test_quantize_of_an_infinity():
    x = torch.ones(4, 256, device="cuda")
    x[2, 5] = float("inf")
    o = _quantize(x, None, h=False, qt=False)
    assert bool(torch.isinf(o["q_sf"][2, 0])) and float(o["q_sf"][2, 1]) == float(torch.tensor(1.0) / 448.0)
    assert bool((o["q"][2, 6:128] == 0).all())


@pytest.mark.parametrize("T,C", [(5, 128), (200, 256), (130, 1024)])
def test_quantize_of_spaced_rows_leaves_the_gaps(T, C):
    g = D.generator(T)
    x, _ = D.spaced(D.randn(g, T, C, dtype=BF16), 24, float("nan"))
    up, _ = D.spaced(D.randn(g, T, C, dtype=BF16), 8, float("nan"))
    h, buf = U.padded(T, C, BF16, 16)
    o = _quantize(x, up, h=False)
    args = dict(num_tokens=T, columns=C, activation=1, scale=1, x=x, up=up, h=h, x_stride=C + 24, up_stride=C + 8, h_stride=C + 16)
    B.mega_moe_quantize(B.make_args(B.mega_moe_quantize_args, **args), U.current_stream())
    v = dense.swiglu(U.f64(x), U.f64(up))
    o["h"] = h
    _check_quantize(o, v, "row", SWIGLU_ROUNDINGS)
    assert bool((buf[:, C:] == 7.0).all())


def _swiglu_backward(x, up, dh, clamp=0.0, grads=True, q=True, qt=True):
    T, C = x.shape
    Tp = D.up128(T)
    both, _ = U.padded(T, 2 * C, x.dtype, 0)
    o = dict(dx=both[:, :C] if grads else None, dup=both[:, C:] if grads else None,
             q=torch.full((T, 2 * C), 0x55, dtype=torch.uint8, device="cuda") if q else None,
             q_sf=torch.full((T, C // 64), 7.0, device="cuda") if q else None,
             qt=torch.full((2 * C, Tp), 0x55, dtype=torch.uint8, device="cuda") if qt else None,
             qt_sf=torch.full((2 * C, Tp // 128), 7.0, device="cuda") if qt else None)
    B.mega_moe_swiglu_backward(B.make_args(
        B.mega_moe_swiglu_backward_args, num_tokens=T, columns=C, x_type=U.TYPE[x.dtype], activation_clamp=clamp, x=x, up=up, dh=dh,
        x_stride=x.stride(0), up_stride=up.stride(0), dh_stride=dh.stride(0), dx_stride=2 * C, dup_stride=2 * C, **o), U.current_stream())
    return o


@pytest.mark.parametrize("T,C", [(1, 128), (5, 2048), (127, 256), (128, 128), (129, 384), (577, 512)])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("clamp", [0.0, 3.0])
def test_swiglu_backward(T, C, dtype, clamp):
    g = D.generator(T * 3 + C)
    both = D.randn(g, T, 2 * C, scale=2.0, dtype=dtype)
    x, up, dh = both[:, :C], both[:, C:], D.randn(g, T, C, scale=1e-2, dtype=dtype)
    full = _swiglu_backward(x, up, dh, clamp)
    dx, dx_mag, dup, dup_mag = dense.swiglu_backward(U.f64(x), U.f64(up), U.f64(dh), clamp)
    # exp, sums, quotient and four products
    n = 16
    U.near(full["dx"], dx, dx_mag, n, "dx")
    U.near(full["dup"], dup, dup_mag, n, "dup")
    v, mag = np.concatenate([dx, dup], axis=1), np.concatenate([dx_mag, dup_mag], axis=1)
    D.check_codes(full["q"], full["q_sf"], dense.rows_quotients(v, mag), n, "q")
    D.check_codes(full["qt"], full["qt_sf"], dense.transposed_quotients(v, mag), n, "qt")
    assert bool((full["qt"][:, T:] == 0).all())
    for kw in (dict(q=False, qt=False), dict(grads=False, qt=False), dict(grads=False, q=False), dict(qt=False)):
        o = _swiglu_backward(x, up, dh, clamp, **kw)
        for name, t in o.items():
            assert t is None or torch.equal(t, full[name]), (kw, name)


def test_swiglu_backward_against_differences():
    g = D.generator(2)
    x, up, dh = (D.randn(g, 3, 128) for _ in range(3))
    o = _swiglu_backward(x, up, dh, q=False, qt=False)
    X, Y, S = U.f64(x), U.f64(up), U.f64(dh)
    e = 1e-5
    dx = (dense.swiglu(X + e, Y) - dense.swiglu(X - e, Y)) / (2 * e) * S
    dup = (dense.swiglu(X, Y + e) - dense.swiglu(X, Y - e)) / (2 * e) * S
    # differences: e^2 / 6 of a third derivative below 2, and float64's rounding over e
    limit = (e * e + 1e-10) * np.abs(S) * (1 + np.abs(Y)) + 24 * U.U * np.abs(S) * (1 + np.abs(X)) * (1 + np.abs(Y))
    assert (np.abs(U.f64(o["dx"]) - dx) <= limit).all() and (np.abs(U.f64(o["dup"]) - dup) <= limit).all()


def test_swiglu_of_extreme_gates_is_finite():
    x = torch.tensor([-3e38, -200.0, -95.0, -88.0, 0.0, -0.0, 88.0, 200.0, 1e30] + [1.0] * 119, device="cuda").repeat(2, 1)
    up = torch.ones_like(x)
    o = _quantize(x, up, qt=False, q=False)
    want = np.clip(dense.swiglu(U.f64(x), U.f64(up)), -3.3e38, 3.3e38)
    U.near(o["h"], want, np.abs(want) + 2.0 ** -120, SWIGLU_ROUNDINGS)
    gr = _swiglu_backward(x, up, torch.ones_like(x))
    assert bool(gr["dx"].isfinite().all()) and bool(gr["dup"].isfinite().all())
    assert float(gr["dx"][0, 0]) == 0.0 and float(gr["dx"][0, 7]) == 1.0


# ---- head norms and rotation -------------------------------------------------------

ROTARY = [  # T, q_heads, k_heads, D, R, start, interleaved, type, weights, far
    (1, 64, 8, 128, 128, 0, False, BF16, True, 1000000), (1, 1, 0, 64, 64, 0, False, F32, True, 0), (3, 2, 1, 8, 0, 0, False, BF16, True, 0),
    (5, 7, 1, 80, 80, 0, False, BF16, True, 0), (33, 9, 3, 96, 48, 0, True, BF16, True, 50000), (100, 4, 4, 192, 64, 128, True, F32, True, 7),
    (257, 3, 2, 256, 128, 0, False, BF16, True, 0), (40, 2, 2, 512, 512, 0, True, BF16, False, 3), (64, 0, 5, 64, 32, 16, False, F32, False, 0),
    (1300, 32, 8, 128, 128, 0, False, BF16, True, 0), (1025, 12, 2, 64, 64, 0, True, F32, False, 900000), (17, 5, 5, 16, 16, 0, False, BF16, True, 0),
    (90, 3, 1, 320, 80, 240, False, F32, True, 0), (4100, 2, 1, 32, 32, 0, False, BF16, True, 0)]


def _rotary_case(T, hq, hk, dim, R, start, interleaved, dtype, weights, far, seed=0, gap=True):
    """Inputs with q and k inside one projection's rows (with gaps between heads), positions and frequencies."""
    g = D.generator(T + hq + dim + seed)
    pitch = dim + (8 if gap else 0)
    c = {"T": T, "hq": hq, "hk": hk, "D": dim}

    def heads(scale, fill=None):
        buf = D.randn(g, T, hq + hk + 1, pitch, scale=scale, dtype=dtype) if fill is None else torch.full((T, hq + hk + 1, pitch), fill, dtype=dtype, device="cuda")
        return buf[:, :hq, :dim], buf[:, hq:hq + hk, :dim], buf

    c["heads"] = heads
    c["q"], c["k"], _ = heads(1.5)
    w = lambda n: (1.0 + D.randn(g, dim, scale=0.2)).to(F32) if weights and n else None   # noqa: E731
    c["q_weight"], c["k_weight"] = w(hq), w(hk)
    c["positions"] = (far + torch.randperm(T, generator=torch.Generator().manual_seed(seed))).to(torch.int32).cuda()
    c["inv_freq"] = torch.tensor([10000.0 ** (-2.0 * i / max(R, 1)) for i in range(R // 2)], dtype=torch.float32, device="cuda")
    c["fields"] = dict(num_tokens=T, q_heads=hq, k_heads=hk, head_dim=dim, rotary_dim=R, rotary_start=start,
                       layout=B.MEGA_MOE_ROTARY_INTERLEAVED if interleaved else B.MEGA_MOE_ROTARY_HALF, type=U.TYPE[dtype],
                       weight_type=B.MEGA_MOE_F32, eps=1e-6, scale=1.25, q_weight=c["q_weight"], k_weight=c["k_weight"],
                       positions=c["positions"], inv_freq=c["inv_freq"])
    c["oracle"] = dict(positions=c["positions"].cpu().numpy(), inv_freq=U.f64(c["inv_freq"]), start=start, interleaved=interleaved,
                       eps=1e-6, scale=1.25)
    return c


def tensors(**named):
    f = {}
    for name, t in named.items():
        if t is not None and t.shape[1]:
            f[name], f[name + "_stride"], f[name + "_head_stride"] = t, t.stride(0), t.stride(1)
    return f


# squares' sum over D in a tree of at most 8 + 6 additions, root, quotient, weight, cos and sin (their own angle's
# rounding: half a turn times 2^-24 is 4 of theirs), two products and a sum
def _rotary_roundings(dim):
    return 40


@pytest.mark.parametrize("case", ROTARY, ids=str)
def test_rotary(case):
    c = _rotary_case(*case)
    qo, ko, buf = c["heads"](0, 7.0)
    B.mega_moe_rotary(B.make_args(B.mega_moe_rotary_args, **c["fields"], **tensors(q=c["q"], k=c["k"], q_out=qo, k_out=ko)), U.current_stream())
    for name, x, w, o in (("q", c["q"], c["q_weight"], qo), ("k", c["k"], c["k_weight"], ko)):
        if x.shape[1]:
            want, mag = dense.rotary(U.f64(x), None if w is None else U.f64(w), **c["oracle"])
            U.near(o, want, mag, _rotary_roundings(c["D"]), name)
    assert bool((buf[:, :, c["D"]:] == 7.0).all()) and bool((buf[:, -1] == 7.0).all())
    # in place, and without positions where they are a run
    fields = dict(c["fields"])
    B.mega_moe_rotary(B.make_args(B.mega_moe_rotary_args, **fields, **tensors(q=c["q"], k=c["k"], q_out=c["q"], k_out=c["k"])), U.current_stream())
    assert torch.equal(c["q"], qo) and torch.equal(c["k"], ko)


def test_rotary_without_positions_counts_from_the_first():
    case = (70, 3, 2, 64, 64, 0, False, F32, True, 0)
    c = _rotary_case(*case)
    outs = []
    for positions, first in ((None, 900), (torch.arange(900, 970, dtype=torch.int32, device="cuda"), 0)):
        qo, ko, _ = c["heads"](0, 0.0)
        fields = dict(c["fields"], positions=positions, first_position=first)
        B.mega_moe_rotary(B.make_args(B.mega_moe_rotary_args, **fields, **tensors(q=c["q"], k=c["k"], q_out=qo, k_out=ko)), U.current_stream())
        outs.append((qo, ko))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("position", [-2 ** 31, -5, 0, 1, 2 ** 31 - 1])
def test_rotary_by_any_32_bit_position(position):
    c = _rotary_case(2, 2, 1, 64, 64, 0, True, F32, False, 0)
    c["positions"].fill_(position)
    c["oracle"]["positions"] = c["positions"].cpu().numpy()
    qo, ko, _ = c["heads"](0, 0.0)
    B.mega_moe_rotary(B.make_args(B.mega_moe_rotary_args, **c["fields"], **tensors(q=c["q"], k=c["k"], q_out=qo, k_out=ko)), U.current_stream())
    want, mag = dense.rotary(U.f64(c["q"]), None, **c["oracle"])
    U.near(qo, want, mag, 40)


def test_rotary_of_zero_and_nan_heads():
    c = _rotary_case(6, 4, 2, 128, 128, 0, False, BF16, True, 0)
    clean, _, _ = c["heads"](0, 0.0)
    kc = torch.empty(6, 2, 128, dtype=BF16, device="cuda")
    c["q"][1, 2] = 0.0
    B.mega_moe_rotary(B.make_args(B.mega_moe_rotary_args, **c["fields"], **tensors(q=c["q"], k=c["k"], q_out=clean, k_out=kc)), U.current_stream())
    assert bool((clean[1, 2] == 0).all())
    c["q"][3, 1, 7] = float("nan")
    out, _, _ = c["heads"](0, 0.0)
    B.mega_moe_rotary(B.make_args(B.mega_moe_rotary_args, **c["fields"], **tensors(q=c["q"], k=c["k"], q_out=out, k_out=kc)), U.current_stream())
    assert bool(out[3, 1].isnan().all())
    out[3, 1] = clean[3, 1]
    assert torch.equal(out, clean)


def _rotary_backward(c, dqo, dko, dq, dk, **more):
    dqw = torch.full((c["D"],), 7.0, device="cuda") if c["q_weight"] is not None else None
    dkw = torch.full((c["D"],), 7.0, device="cuda") if c["k_weight"] is not None else None
    fields = dict(c["fields"], dq_weight=dqw, dk_weight=dkw)
    fields.update(more)
    a = B.make_args(B.mega_moe_rotary_backward_args, **fields, **tensors(q=c["q"], k=c["k"], dq_out=dqo, dk_out=dko, dq=dq, dk=dk))
    B.set_args(a, **U.workspace(B.mega_moe_rotary_workspace_bytes(a)))
    B.mega_moe_rotary_backward(a, U.current_stream())
    return dqw, dkw


@pytest.mark.parametrize("case", ROTARY, ids=str)
def test_rotary_backward(case):
    c = _rotary_case(*case)
    dqo, dko, _ = c["heads"](0.5)
    dq, dk, buf = c["heads"](0, 7.0)
    dqw, dkw = _rotary_backward(c, dqo, dko, dq, dk)
    for name, x, w, d, dx, dw in (("q", c["q"], c["q_weight"], dqo, dq, dqw), ("k", c["k"], c["k_weight"], dko, dk, dkw)):
        if not x.shape[1]:
            continue
        want, mag, want_w, mag_w = dense.rotary_backward(U.f64(x), None if w is None else U.f64(w), U.f64(d), **c["oracle"])
        U.near(dx, want, mag, 64, "d" + name)
        if w is not None:
            # a thread's run of items, 32 groups at most, a column of 16 rows and 64 of their sums
            U.near(dw, want_w, mag_w, 64 + c["T"] * x.shape[1] // 16 + 128, "weight of " + name)
    assert bool((buf[:, :, c["D"]:] == 7.0).all()) and bool((buf[:, -1] == 7.0).all())
    again = _rotary_backward(c, dqo, dko, dqo, dko)           # in place
    assert torch.equal(dqo, dq) and torch.equal(dko, dk)
    assert all(a is None or torch.equal(a, b) for a, b in zip(again, (dqw, dkw)))


def test_rotary_backward_of_one_weight_alone():
    c = _rotary_case(50, 4, 2, 64, 32, 0, False, F32, True, 0)
    dqo, dko, _ = c["heads"](0.5)
    both = _rotary_backward(c, dqo, dko, *c["heads"](0, 7.0)[:2])
    dq, dk, _ = c["heads"](0, 7.0)
    _, alone = _rotary_backward(c, dqo, dko, dq, dk, dq_weight=None)
    assert torch.equal(alone, both[1])


def test_rotary_backward_without_tokens_clears_the_sums():
    c = _rotary_case(4, 2, 2, 64, 64, 0, False, BF16, True, 0)
    c["fields"]["num_tokens"] = 0
    w = [torch.full((64,), 7.0, device="cuda") for _ in range(2)]
    a = B.make_args(B.mega_moe_rotary_backward_args, **dict(c["fields"], dq_weight=w[0], dk_weight=w[1]))
    B.mega_moe_rotary_backward(a, U.current_stream())
    assert bool((w[0] == 0).all()) and bool((w[1] == 0).all())


def test_rotary_gradients_against_differences():
    c = _rotary_case(2, 2, 1, 32, 16, 8, True, F32, True, 11)
    dqo, dko, _ = c["heads"](0.5)
    dq, dk, _ = c["heads"](0, 0.0)
    dqw, _ = _rotary_backward(c, dqo, dko, dq, dk)
    x, w, d, e = U.f64(c["q"]), U.f64(c["q_weight"]), U.f64(dqo), 1e-5
    loss = lambda x, w: float((dense.rotary(x, w, **c["oracle"])[0] * d).sum())   # noqa: E731
    for at in np.ndindex(*x.shape):
        s = np.zeros_like(x)
        s[at] = e
        # second differences of the norm below 100 at these sizes, float64 over e, float32's roundings
        assert abs((loss(x + s, w) - loss(x - s, w)) / (2 * e) - U.f64(dq)[at]) <= 100 * e * e + 1e-9 + 200 * U.U
    for i in range(32):
        s = np.zeros(32)
        s[i] = e
        assert abs((loss(x, w + s) - loss(x, w - s)) / (2 * e) - U.f64(dqw)[i]) <= 1e-9 + 200 * U.U


def test_rotary_beyond_32_bit_offsets():
    T, dim, stride = 1100, 64, 1 << 21
    c = _rotary_case(T, 2, 1, dim, dim, 0, False, BF16, True, 0, gap=False)
    far = torch.empty((T - 1) * stride + 3 * dim, dtype=BF16, device="cuda")
    q, k = far.as_strided((T, 2, dim), (stride, dim, 1)), far.as_strided((T, 1, dim), (stride, dim, 1), 2 * dim)
    q.copy_(c["q"])
    k.copy_(c["k"])
    B.mega_moe_rotary(B.make_args(B.mega_moe_rotary_args, **c["fields"], **tensors(q=q, k=k, q_out=q, k_out=k)), U.current_stream())
    want, mag = dense.rotary(U.f64(c["q"]), U.f64(c["q_weight"]), **c["oracle"])
    U.near(q.contiguous(), want, mag, 40)
    want, mag = dense.rotary(U.f64(c["k"]), U.f64(c["k_weight"]), **c["oracle"])
    U.near(k.contiguous(), want, mag, 40)
