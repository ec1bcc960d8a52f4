"""The dense path's operators at the limits of their arguments: codes next to
the ties between two of them, offsets beyond 32 bits, memory behind the last
row, tensors that the device does not know."""

import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from oracle import dense
from tests import block_util as U
from tests import dense_util as D

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
u8 = torch.uint8


def _quantize(x, q=None, q_sf=None, qt=None, qt_sf=None, scale="row", **more):
    f = dict(num_tokens=x.shape[0], columns=x.shape[1], x_type=U.TYPE[x.dtype], scale=D.SCALE[scale], x=x, x_stride=x.stride(0),
             q=q, q_sf=q_sf, qt=qt, qt_sf=qt_sf)
    f.update(more)
    B.mega_moe_quantize(B.make_args(B.mega_moe_quantize_args, **f), U.current_stream())


def _new(*shape, dtype=F32, fill=7):
    return torch.full(shape, fill, dtype=dtype, device="cuda")


# ---- codes next to ties -------------------------------------------------------------------------

def _next_to_ties(scales, seed):
    """Blocks of 128 floats of the given scales: the largest is 448 scales, the others lie within
    a few floats of the middle between two codes."""
    g = torch.Generator()
    g.manual_seed(seed)
    codes = torch.arange(0, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    ties = (codes[1:] + codes[:-1]) / 2
    n = scales.numel()
    v = ties[torch.randint(0, ties.numel(), (n, 128), generator=g)] * scales[:, None].double()
    off = torch.randint(-3, 4, (n, 128), generator=g).to(torch.int32)
    x = (v.float().view(torch.int32) + off).view(torch.float32)
    x = x * (1 - 2 * torch.randint(0, 2, (n, 128), generator=g))
    x[:, 0] = 448.0 * scales
    return x


@pytest.mark.parametrize("way", ["rows", "columns", "blocks"])
def test_codes_are_those_of_the_quotient(way):
    # E4M3 of (the value over its float32 scale, rounded to float32): in one code of the two where the middle lies
    g = torch.Generator()
    g.manual_seed(2)
    scales = torch.rand(2048, generator=g) + 0.5 if way != "blocks" else (torch.rand(16, generator=g) + 0.5).repeat_interleave(128)
    scales = scales * torch.exp2(torch.randint(-110, 100, (scales.numel() // 128,), generator=g).float()).repeat_interleave(128)
    x = _next_to_ties(scales, 3)                         # [2048, 128]
    q, q_sf, qt, qt_sf = _new(2048, 128, dtype=u8), _new(2048, 1), _new(128, 2048, dtype=u8), _new(128, 16)
    if way == "columns":
        # the blocks as columns: [16 x 128 tokens, 128 columns]
        src = x.view(16, 128, 128).transpose(1, 2).reshape(2048, 128).contiguous()
        _quantize(src.cuda(), qt=qt, qt_sf=qt_sf)
        got = qt.cpu().view(128, 16, 128).permute(1, 0, 2).reshape(2048, 128)
        sf = qt_sf.cpu().t().reshape(2048, 1)
    elif way == "blocks":
        q_sf = _new(16, 1)
        _quantize(x.cuda(), q=q, q_sf=q_sf, scale="block")
        got, sf = q.cpu(), q_sf.cpu().repeat_interleave(128, dim=0)
    else:
        _quantize(x.cuda(), q=q, q_sf=q_sf)
        got, sf = q.cpu(), q_sf.cpu()
    most = x.abs().amax(dim=1, keepdim=True) if way != "blocks" else x.abs().view(16, -1).amax(dim=1).repeat_interleave(128)[:, None]
    assert torch.equal(sf, most / 448.0)
    want = (x.double() / sf.double()).float().to(torch.float8_e4m3fn).view(u8)
    assert torch.equal(got, want), int((got != want).sum())


# ---- offsets beyond 32 bits ---------------------------------------------------------------------

def test_codes_beyond_32_bit_offsets():
    T, C = (1 << 21) - 3, 2048                           # 4.3e9 values
    g = D.generator(3)
    x = torch.zeros(T, C, dtype=BF16, device="cuda")
    tail = 256 + 125                                     # whole blocks of rows, and the last
    x[-tail:] = D.randn(g, tail, C, dtype=BF16)
    x[:128] = D.randn(g, 128, C, dtype=BF16)
    Tp = D.up128(T)
    q, q_sf = torch.empty(T, C, dtype=u8, device="cuda"), torch.empty(T, C // 128, device="cuda")
    qt, qt_sf = torch.empty(C, Tp, dtype=u8, device="cuda"), torch.empty(C, Tp // 128, device="cuda")
    _quantize(x, q, q_sf, qt, qt_sf)
    assert (T - tail) % 128 == 0
    for part, at in ((x[-tail:], slice(T - tail, Tp)), (x[:128], slice(0, 128))):
        rows = slice(at.start, at.start + part.shape[0])
        v = U.f64(part)
        D.check_codes(q[rows], q_sf[rows], dense.rows_quotients(v), 4, "q")
        D.check_codes(qt[:, at].contiguous(), qt_sf[:, at.start // 128:at.stop // 128].contiguous(), dense.transposed_quotients(v), 4, "qt")
    # between them all is zero
    assert not bool(q[128:T - tail].any()) and not bool(q_sf[128:T - tail].any()) and not bool(qt_sf[:, 1:(T - tail) // 128].any())
    del qt, qt_sf
    _quantize(x, q, q_sf)                                # the kernel for rows alone
    D.check_codes(q[-tail:], q_sf[-tail:], dense.rows_quotients(U.f64(x[-tail:])), 4, "q alone")


def test_gradients_beyond_32_bit_offsets():
    T, C, stride = 1100, 128, 1 << 22
    g = D.generator(6)
    far = torch.empty((T - 1) * stride + 3 * C, dtype=BF16, device="cuda")
    x, up, dh = (far.as_strided((T, C), (stride, 1), i * C) for i in range(3))
    for t, s in ((x, 2.0), (up, 2.0), (dh, 0.01)):
        t.copy_(D.randn(g, T, C, scale=s, dtype=BF16))
    wide = torch.empty((T - 1) * stride + 2 * C, dtype=BF16, device="cuda")
    dx, dup = (wide.as_strided((T, C), (stride, 1), i * C) for i in range(2))
    B.mega_moe_swiglu_backward(B.make_args(B.mega_moe_swiglu_backward_args, num_tokens=T, columns=C, x_type=B.MEGA_MOE_BF16, x=x, up=up, dh=dh,
                                           dx=dx, dup=dup, x_stride=stride, up_stride=stride, dh_stride=stride, dx_stride=stride,
                                           dup_stride=stride), U.current_stream())
    want = dense.swiglu_backward(*(U.f64(t.contiguous()) for t in (x, up, dh)))
    U.near(dx.contiguous(), want[0], want[1], 16, "dx")
    U.near(dup.contiguous(), want[2], want[3], 16, "dup")


def test_head_gradients_beyond_32_bit_offsets():
    T, dim, stride = 1100, 64, 1 << 22
    g = D.generator(7)
    far = torch.empty((T - 1) * stride + 4 * dim, dtype=BF16, device="cuda")
    q, dq = far.as_strided((T, 2, dim), (stride, dim, 1)), far.as_strided((T, 2, dim), (stride, dim, 1), 2 * dim)
    q.copy_(D.randn(g, T, 2, dim, dtype=BF16))
    d = D.randn(g, T, 2, dim, dtype=BF16)
    dq.copy_(d)
    weight, freq, dw = 1 + D.randn(g, dim, scale=0.1), torch.tensor([10000.0 ** (-i / 32) for i in range(32)], device="cuda"), _new(dim)
    args = B.make_args(B.mega_moe_rotary_backward_args, num_tokens=T, q_heads=2, head_dim=dim, rotary_dim=dim, weight_type=B.MEGA_MOE_F32,
                       eps=1e-6, q=q, q_weight=weight, inv_freq=freq, dq_out=dq, dq=dq, dq_weight=dw, q_stride=stride, dq_out_stride=stride,
                       dq_stride=stride)
    B.set_args(args, **U.workspace(B.mega_moe_rotary_workspace_bytes(args)))
    B.mega_moe_rotary_backward(args, U.current_stream())
    want = dense.rotary_backward(U.f64(q.contiguous()), U.f64(weight), U.f64(d), range(T), U.f64(freq), eps=1e-6)
    U.near(dq.contiguous(), want[0], want[1], 96, "dq")
    U.near(dw, want[2], want[3], 96 + 2 * T, "dw")


# ---- heads of q, k and v in turn ----------------------------------------------------------------

@pytest.mark.parametrize("T", [1, 37, 600])
def test_heads_in_turn_are_turned_in_place(T):
    g = D.generator(T)
    heads, dim = 5, 64
    buf = D.randn(g, T, heads, 3, dim, dtype=BF16)
    first, d = buf.clone(), D.randn(g, T, heads, 3, dim, dtype=BF16)
    grads = d.clone()
    weight = 1 + D.randn(g, dim, scale=0.1)
    freq = torch.tensor([10000.0 ** (-i / 32) for i in range(32)], device="cuda")
    dw = _new(2, dim)
    f = dict(num_tokens=T, q_heads=heads, k_heads=heads, head_dim=dim, rotary_dim=dim, weight_type=B.MEGA_MOE_F32, eps=1e-6, inv_freq=freq,
             q_weight=weight, k_weight=weight)
    names = lambda *n: {k: v for name in n for k, v in ((name + "_stride", 3 * heads * dim), (name + "_head_stride", 3 * dim))}   # noqa: E731
    q, k = buf[:, :, 0], buf[:, :, 1]
    B.mega_moe_rotary(B.make_args(B.mega_moe_rotary_args, q=q, k=k, q_out=q, k_out=k, **f, **names("q", "k", "q_out", "k_out")),
                      U.current_stream())
    dq, dk, x = grads[:, :, 0], grads[:, :, 1], first
    args = B.make_args(B.mega_moe_rotary_backward_args, q=x[:, :, 0], k=x[:, :, 1], dq_out=dq, dk_out=dk, dq=dq, dk=dk, dq_weight=dw[0],
                       dk_weight=dw[1], **f, **names("q", "k", "dq_out", "dk_out", "dq", "dk"))
    B.set_args(args, **U.workspace(B.mega_moe_rotary_workspace_bytes(args)))
    B.mega_moe_rotary_backward(args, U.current_stream())
    for i in range(2):
        x = U.f64(first[:, :, i])
        want, mag = dense.rotary(x, U.f64(weight), range(T), U.f64(freq), eps=1e-6)
        U.near(buf[:, :, i], want, mag, 40, f"heads {i}")
        want = dense.rotary_backward(x, U.f64(weight), U.f64(d[:, :, i]), range(T), U.f64(freq), eps=1e-6)
        U.near(grads[:, :, i], want[0], want[1], 96, f"gradients {i}")
        U.near(dw[i], want[2], want[3], 96 + heads * T, f"weight {i}")
    assert torch.equal(buf[:, :, 2], first[:, :, 2]) and torch.equal(grads[:, :, 2], d[:, :, 2])


# ---- memory behind the last row -----------------------------------------------------------------

@pytest.mark.parametrize("m", [1, 13, 61, 129, 300])
def test_memory_behind_the_outputs_stays(m):
    g = D.generator(m)
    k, n = 256, 200
    a, a_sf = D.operand(g, m, k)
    b, b_sf = D.operand(g, n, k, "block")
    for out_type in (BF16, F32):
        out = _new(m + 9, n, dtype=out_type)
        D.product(a, a_sf, b, b_sf, out[:m], "block")
        assert bool((out[m:] == 7).all()) and not bool((out[:m] == 7).all())
    x, up, dh = (D.randn(g, m, k, dtype=BF16) for _ in range(3))
    Tp = D.up128(m)
    for two in (False, True):
        rows = 2 * k if two else k
        q, q_sf = _new(m + 9, rows, dtype=u8), _new(m + 9, rows // 128)
        qt, qt_sf = _new(rows + 9, Tp, dtype=u8), _new(rows + 9, Tp // 128)
        if two:
            B.mega_moe_swiglu_backward(B.make_args(B.mega_moe_swiglu_backward_args, num_tokens=m, columns=k, x_type=B.MEGA_MOE_BF16, x=x, up=up,
                                                   dh=dh, q=q, q_sf=q_sf, qt=qt, qt_sf=qt_sf), U.current_stream())
        else:
            _quantize(x, q, q_sf, qt, qt_sf)
        for t, end in ((q, m), (q_sf, m), (qt, rows), (qt_sf, rows)):
            assert bool((t[end:] == 7).all()) and not bool((t[:end] == 7).all())
    heads, dim = 3, 48
    h, freq = D.randn(g, m, heads, dim), torch.rand(dim // 2, device="cuda", generator=g)
    out, w = _new(m + 9, heads, dim), torch.ones(dim, device="cuda")
    B.mega_moe_rotary(B.make_args(B.mega_moe_rotary_args, num_tokens=m, q_heads=heads, head_dim=dim, rotary_dim=dim, type=B.MEGA_MOE_F32,
                                  weight_type=B.MEGA_MOE_F32, eps=1e-6, q=h, q_weight=w, inv_freq=freq, q_out=out), U.current_stream())
    assert bool((out[m:] == 7).all())
    d, dq, dw = out[:m].clone(), _new(m + 9, heads, dim), _new(dim + 9)
    args = B.make_args(B.mega_moe_rotary_backward_args, num_tokens=m, q_heads=heads, head_dim=dim, rotary_dim=dim, type=B.MEGA_MOE_F32,
                       weight_type=B.MEGA_MOE_F32, eps=1e-6, q=h, q_weight=w, inv_freq=freq, dq_out=d, dq=dq, dq_weight=dw)
    need = B.mega_moe_rotary_workspace_bytes(args)
    ws = _new(need + 64, dtype=u8)
    B.set_args(args, workspace=ws, workspace_bytes=need)
    B.mega_moe_rotary_backward(args, U.current_stream())
    assert bool((dq[m:] == 7).all()) and bool((dw[dim:] == 7).all()) and bool((ws[need:] == 7).all())


def test_memory_behind_the_partial_sums_stays():
    g = D.generator(1)
    m, k, n = 136, 16384, 144
    a, a_sf = D.operand(g, m, k)
    b, b_sf = D.operand(g, n, k)
    out = _new(m, n)
    args = D.product_args(a, a_sf, b, b_sf, out, "row")
    need = B.mega_moe_product_workspace_bytes(args)
    ws = _new(need + 64, dtype=u8)
    B.set_args(args, workspace=ws, workspace_bytes=need)
    B.mega_moe_product(args, U.current_stream())
    D.check_product(out, a, a_sf, b, b_sf, "row")
    assert need > 0 and bool((ws[need:] == 7).all())


# ---- tensors that the device does not know --------------------------------------------------------

def test_a_first_tensor_in_host_memory_is_refused():
    T, C = 4, 256
    rows, heads = torch.zeros(T, C, dtype=BF16, device="cuda"), torch.zeros(T, 2, 64, dtype=BF16, device="cuda")
    codes, sf, out = _new(T, C, dtype=u8, fill=0), _new(T, C // 128, fill=0), _new(T, 8, dtype=BF16)
    b, b_sf, freq = _new(8, C, dtype=u8, fill=0), _new(1, C // 128, fill=0), torch.zeros(32, device="cuda")
    norm = dict(num_tokens=T, q_heads=2, head_dim=64, rotary_dim=64, inv_freq=freq)
    calls = [
        (B.mega_moe_product, B.mega_moe_product_args, "a", codes, dict(m=T, n=8, k=C, a_sf=sf, b=b, b_sf=b_sf, out=out)),
        (B.mega_moe_product, B.mega_moe_product_args, "out", out, dict(m=T, n=8)),
        (B.mega_moe_quantize, B.mega_moe_quantize_args, "x", rows, dict(num_tokens=T, columns=C, scale=1, q=codes, q_sf=sf)),
        (B.mega_moe_swiglu_backward, B.mega_moe_swiglu_backward_args, "x", rows,
         dict(num_tokens=T, columns=C, up=rows, dh=rows, dx=torch.zeros_like(rows))),
        (B.mega_moe_rotary, B.mega_moe_rotary_args, "q", heads, dict(q_out=torch.zeros_like(heads), **norm)),
        (B.mega_moe_rotary_backward, B.mega_moe_rotary_backward_args, "dq_out", heads, dict(dq=torch.zeros_like(heads), **norm)),
    ]
    for call, cls, first, good, others in calls:
        a = B.make_args(cls, **{first: good}, **others)
        assert call(a, U.current_stream()) == 0, call.__name__
        # aligned as a device's tensor is, in ordinary memory: the refusal is the host's
        host = torch.zeros(good.numel() * good.element_size() + 64, dtype=u8)
        B.set_args(a, **{first: host.data_ptr() + -host.data_ptr() % 64})
        with pytest.raises(B.MegaMoEError) as ei:
            call(a, U.current_stream())
        assert ei.value.code == B.MEGA_MOE_ERR_INVALID_ARG and "host memory" in B.mega_moe_last_error()
    torch.cuda.synchronize()
