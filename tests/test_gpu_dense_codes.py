"""E4M3 codes of mega_moe_quantize where scales are far from 1: those next to
the smallest float32 numbers, rounded or lost, and those next to the largest."""

import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from tests.test_gpu_dense_limits import _new, _next_to_ties, _quantize

pytestmark = pytest.mark.gpu

u8 = torch.uint8


def _codes(x, way):
    """Codes and scales of x [rows, 128], a block to a row ("blocks": to 128 rows), by the kernel's three ways."""
    rows = x.shape[0]
    if way == "columns":
        # the blocks as columns: [rows / 128 x 128 tokens, 128 columns]
        src = x.view(-1, 128, 128).transpose(1, 2).reshape(rows, 128).contiguous()
        qt, qt_sf = _new(128, rows, dtype=u8), _new(128, rows // 128)
        _quantize(src.cuda(), qt=qt, qt_sf=qt_sf)
        return qt.cpu().view(128, -1, 128).permute(1, 0, 2).reshape(rows, 128), qt_sf.cpu().t().reshape(rows, 1)
    if way == "blocks":
        q, q_sf = _new(rows, 128, dtype=u8), _new(rows // 128, 1)
        _quantize(x.cuda(), q=q, q_sf=q_sf, scale="block")
        return q.cpu(), q_sf.cpu().repeat_interleave(128, dim=0)
    q, q_sf = _new(rows, 128, dtype=u8), _new(rows, 1)
    more = dict(qt=_new(128, rows, dtype=u8), qt_sf=_new(128, rows // 128)) if way == "both" else {}
    _quantize(x.cuda(), q=q, q_sf=q_sf, **more)
    return q.cpu(), q_sf.cpu()


def _most(x, way):
    return x.abs().amax(dim=1, keepdim=True) if way != "blocks" else x.abs().view(-1, 128 * 128).amax(dim=1).repeat_interleave(128)[:, None]


def _want(x, sf):
    """The quotient rounded to float32, then to E4M3, at most its largest value; 0 where the scale is."""
    quotient = (x.double() / sf.double()).float()
    return torch.where(sf > 0, quotient.clamp(-448.0, 448.0), torch.zeros(())).to(torch.float8_e4m3fn).view(u8)


def _same(got, want):
    """The same codes; of a 0 the sign is of no matter."""
    off = (got != want) & (((got | want) & 0x7F) != 0)
    assert not bool(off.any()), int(off.sum())


def _scales(rows, lo, hi, way, g):
    n = rows // 128 if way == "blocks" else rows
    s = (torch.rand(n, generator=g).double() + 0.5) * torch.exp2(torch.randint(lo, hi + 1, (n,), generator=g).double())
    return s.repeat_interleave(rows // n)


WAYS = ["rows", "both", "columns", "blocks"]


@pytest.mark.parametrize("way", WAYS)
def test_codes_of_subnormal_scales_are_those_of_the_quotient(way):
    g = torch.Generator()
    g.manual_seed(5)
    # the scale before it is rounded, from below half the smallest float up to the normal ones
    scales = _scales(8192, -151, -124, way, g)
    x = ((2 * torch.rand(8192, 128, generator=g).double() - 1) * 448 * scales[:, None]).float()
    x[:, 0] = (448 * scales).float()
    got, sf = _codes(x, way)
    # float64's quotient of a float32 number, rounded to a subnormal float32: a float32 division's own
    assert torch.equal(sf, (_most(x, way).double() / 448.0).float())
    assert bool((sf == 0).any()) and bool((sf == 2.0 ** -149).any()) and bool((sf > 2.0 ** -126).any())
    _same(got, _want(x, sf))


@pytest.mark.parametrize("way", WAYS)
def test_codes_of_the_largest_scales_are_those_of_the_quotient(way):
    g = torch.Generator()
    g.manual_seed(6)
    x = _next_to_ties(_scales(16384, 100, 118, way, g).float(), 7)
    got, sf = _codes(x, way)
    assert torch.equal(sf, _most(x, way) / 448.0) and bool(sf.isfinite().all())
    _same(got, _want(x, sf))


@pytest.mark.parametrize("way", WAYS)
def test_codes_where_scales_of_all_sizes_meet(way):
    # tiny, ordinary and large blocks side by side, in one wave's rows and columns
    g = torch.Generator()
    g.manual_seed(8)
    exponents = torch.tensor([-130.0, -127.0, -101.0, -99.0, -3.0, 0.0, 60.0, 63.0, 64.0, 65.0, 110.0, 118.0])
    n = 32 if way == "blocks" else 4096
    scales = (torch.rand(n, generator=g) + 0.5) * torch.exp2(exponents[torch.randint(0, len(exponents), (n,), generator=g)])
    x = _next_to_ties(scales.repeat_interleave(4096 // n), 9)
    got, sf = _codes(x, way)
    assert torch.equal(sf, (_most(x, way).double() / 448.0).float())
    _same(got, _want(x, sf))


def test_gradients_codes_of_subnormal_scales():
    # gate 0 gives dx = dh * up / 2 and dup = 0, exact: the codes by rows and by columns of dx
    g = torch.Generator()
    g.manual_seed(10)
    x = torch.zeros(256, 128)
    scales = _scales(256, -150, -126, "rows", g)
    dh = ((2 * torch.rand(256, 128, generator=g).double() - 1) * 448 * scales[:, None]).float()
    q, q_sf, qt, qt_sf = _new(256, 256, dtype=u8), _new(256, 2), _new(256, 256, dtype=u8), _new(256, 2)
    B.mega_moe_swiglu_backward(B.make_args(
        B.mega_moe_swiglu_backward_args, num_tokens=256, columns=128, x_type=B.MEGA_MOE_F32, x=x.cuda(), up=torch.full_like(x, 2.0).cuda(),
        dh=dh.cuda(), q=q, q_sf=q_sf, qt=qt, qt_sf=qt_sf), torch.cuda.current_stream().cuda_stream)
    for v, codes, sf in ((dh, q[:, :128], q_sf[:, :1]), (dh.t(), qt[:128], qt_sf[:128])):
        codes, sf = codes.cpu(), sf.cpu()
        blocks = v.reshape(v.shape[0], -1, 128)
        assert torch.equal(sf, (blocks.abs().amax(dim=2).double() / 448.0).float())
        _same(codes, _want(blocks, sf[:, :, None]).reshape(v.shape))
    assert not bool((q[:, 128:] & 0x7F).any()) and not bool(q_sf[:, 1].any())
