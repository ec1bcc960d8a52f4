"""The dense path's operators in a run, as a block with attention's projections
and a shared expert beside the routed ones trains with them: the norm makes the
E4M3 rows; the projections' product, the heads' norms and rotation; the layer,
and beside it the shared expert's two products around the activation, added to
the layer's output; then the gradients of both, with the weights' gradients
added to those of earlier tokens.  Each step is checked against the float64
reference on the values that the step before it gave; then the whole run again
on another stream, from a captured graph with eager work between its replays,
and two captured runs at once.
"""

import numpy as np
import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from fp8_mixture_experts_amd import synthetic as S
from oracle import dense, moe
from tests import block_util as U
from tests import dense_util as D
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
T, H, I, E, K = 61, 512, 256, 16, 4
HQ, HK, DIM = 4, 2, 64
N = (HQ + 2 * HK) * DIM              # q, k and v beside each other
EPS = 1e-6


class Run:
    def __init__(self, seed, tokens=T):
        g = D.generator(seed)
        r = lambda *s, dtype=F32, scale=1.0: D.randn(g, *s, scale=scale, dtype=dtype)   # noqa: E731
        new = lambda *s, dtype=F32: torch.zeros(s, dtype=dtype, device="cuda")   # noqa: E731
        u8 = torch.uint8
        tp = D.up128(tokens)
        self.tokens = tokens
        self.weights = S.make_weights(S.custom(tokens=tokens, hidden=H, intermediate=I, experts=E, topk=K, weight_seed=5))
        self.dev = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in self.weights.items()}
        self.layer = B.MegaMoE(E, H, I, K, tokens)
        self.args = []
        # the weights, by blocks, both ways; once, as a step that has changed them would
        self.w = {}
        for name, rows, cols in (("qkv", N, H), ("gate_up", 2 * I, H), ("down", H, I)):
            x = r(rows, cols, dtype=BF16, scale=cols ** -0.5)
            w = dict(q=new(rows, cols, dtype=u8), q_sf=new(rows // 128, cols // 128), qt=new(cols, rows, dtype=u8),
                     qt_sf=new(cols // 128, rows // 128))
            B.mega_moe_quantize(B.make_args(B.mega_moe_quantize_args, num_tokens=rows, columns=cols, x_type=B.MEGA_MOE_BF16,
                                            scale=B.MEGA_MOE_SCALE_BLOCK, x=x, **w), U.current_stream())
            self.w[name] = w
        # inputs
        self.h, self.pre = r(tokens, H, dtype=BF16), 1 + r(H, scale=0.1)
        self.idx = torch.rand(tokens, E, generator=g, device="cuda").argsort(dim=1)[:, :K].to(torch.int32).contiguous()
        self.weight = torch.rand(tokens, K, generator=g, device="cuda")
        self.q_weight, self.k_weight = 1 + r(DIM, scale=0.1), 1 + r(DIM, scale=0.1)
        self.positions = torch.randint(0, 5000, (tokens,), generator=g, device="cuda", dtype=torch.int32)
        host = torch.empty(DIM // 2)
        B.mega_moe_rotary_frequencies(B.make_args(B.mega_moe_rotary_frequencies_args, rotary_dim=DIM,
                                                  scaling=B.MEGA_MOE_ROTARY_PLAIN, base=10000.0, inv_freq=host))
        self.inv_freq = host.cuda()
        self.dy, self.dqkv_out = r(tokens, H, dtype=BF16, scale=0.01), r(tokens, N, dtype=BF16, scale=0.01)
        self.before = {"qkv": r(N, H, scale=0.1), "gate_up": r(2 * I, H, scale=0.1), "down": r(H, I, scale=0.1)}
        # outputs
        self.n, self.q, self.q_sf = new(tokens, H, dtype=BF16), new(tokens, H, dtype=u8), new(tokens, H // 128)
        self.nt, self.nt_sf = new(H, tp, dtype=u8), new(H, tp // 128)
        self.qkv, self.turned, self.gate_up = new(tokens, N, dtype=BF16), new(tokens, N, dtype=BF16), new(tokens, 2 * I, dtype=BF16)
        self.a, self.a_sf, self.at, self.at_sf = new(tokens, I, dtype=u8), new(tokens, I // 128), new(I, tp, dtype=u8), new(I, tp // 128)
        self.routed, self.y = new(tokens, H, dtype=BF16), new(tokens, H, dtype=BF16)
        self.dyq, self.dyq_sf, self.dyt, self.dyt_sf = new(tokens, H, dtype=u8), new(tokens, H // 128), new(H, tp, dtype=u8), new(H, tp // 128)
        self.da = new(tokens, I, dtype=BF16)
        self.dgq, self.dgq_sf = new(tokens, 2 * I, dtype=u8), new(tokens, 2 * I // 128)
        self.dgt, self.dgt_sf = new(2 * I, tp, dtype=u8), new(2 * I, tp // 128)
        self.dn0, self.dn = new(tokens, H, dtype=BF16), new(tokens, H, dtype=BF16)
        self.dqkv, self.dq_weight, self.dk_weight = new(tokens, N, dtype=BF16), new(DIM), new(DIM)
        self.dpq, self.dpq_sf, self.dpt, self.dpt_sf = new(tokens, N, dtype=u8), new(tokens, N // 128), new(N, tp, dtype=u8), new(N, tp // 128)
        self.dw = {k: torch.zeros_like(v) for k, v in self.before.items()}

        self.steps = []
        self._norm()
        self._product("qkv", self.q, self.q_sf, self.w["qkv"], self.qkv)
        self._rotary()
        self._product("gate_up", self.q, self.q_sf, self.w["gate_up"], self.gate_up)
        self._quantize(I, self.gate_up[:, :I], self.gate_up[:, I:], q=self.a, q_sf=self.a_sf, qt=self.at, qt_sf=self.at_sf)
        self._add(lambda s: B.mega_moe_forward(self.layer.handle, tokens, self.q, self.q_sf, self.idx, self.weight, self.dev["w1"],
                                               self.dev["w1_sf"], self.dev["w2"], self.dev["w2_sf"], self.routed, s))
        self._product("down", self.a, self.a_sf, self.w["down"], self.y, add=self.routed)
        # gradients of the shared expert
        self._quantize(H, self.n, qt=self.nt, qt_sf=self.nt_sf)
        self._quantize(H, self.dy, q=self.dyq, q_sf=self.dyq_sf, qt=self.dyt, qt_sf=self.dyt_sf)
        self._gradients("down", self.dyq, self.dyq_sf, self.dyt, self.dyt_sf, self.at, self.at_sf, self.da)
        args = B.make_args(B.mega_moe_swiglu_backward_args, num_tokens=tokens, columns=I, x_type=B.MEGA_MOE_BF16, x=self.gate_up[:, :I],
                           up=self.gate_up[:, I:], dh=self.da, q=self.dgq, q_sf=self.dgq_sf, qt=self.dgt, qt_sf=self.dgt_sf,
                           x_stride=2 * I, up_stride=2 * I)
        self._add(lambda s: B.mega_moe_swiglu_backward(args, s))
        self._gradients("gate_up", self.dgq, self.dgq_sf, self.dgt, self.dgt_sf, self.nt, self.nt_sf, self.dn0)
        # and of the projections, whose gradient of the rows is added to it
        self._rotary_backward()
        self._quantize(N, self.dqkv, q=self.dpq, q_sf=self.dpq_sf, qt=self.dpt, qt_sf=self.dpt_sf)
        self._gradients("qkv", self.dpq, self.dpq_sf, self.dpt, self.dpt_sf, self.nt, self.nt_sf, self.dn, add=self.dn0)

    OUT = ("n", "q", "q_sf", "nt", "nt_sf", "qkv", "turned", "gate_up", "a", "a_sf", "at", "at_sf", "routed", "y", "dyq", "dyq_sf",
           "dyt", "dyt_sf", "da", "dgq", "dgq_sf", "dgt", "dgt_sf", "dn0", "dn", "dqkv", "dq_weight", "dk_weight", "dpq", "dpq_sf",
           "dpt", "dpt_sf")

    def _add(self, step):
        self.steps.append(step)

    def _norm(self):
        args = B.make_args(B.mega_moe_norm_args, num_tokens=self.tokens, hidden=H, weight_type=B.MEGA_MOE_F32, gate_type=B.MEGA_MOE_F32,
                           residual_scale=1.0, pre_eps=EPS, post_eps=EPS, h=self.h, pre_weight=self.pre, n=self.n, q=self.q, q_sf=self.q_sf)
        self._add(lambda s: B.mega_moe_norm(args, s))

    def _product(self, name, a, a_sf, w, out, add=None):
        args = D.product_args(a, a_sf, w["q"], w["q_sf"], out, "block", add)
        self._add(lambda s: B.mega_moe_product(args, s))

    def _gradients(self, name, dq, dq_sf, dt, dt_sf, xt, xt_sf, dx, add=None):
        """dx = dout . w (the transposed codes), dw = before + dout^T . x."""
        w = self.w[name]
        first = D.product_args(dq, dq_sf, w["qt"], w["qt_sf"], dx, "block", add)
        second = D.product_args(dt, dt_sf, xt, xt_sf, self.dw[name], "row", self.before[name])
        self._add(lambda s: B.mega_moe_product(first, s))
        self._add(lambda s: B.mega_moe_product(second, s))

    def _quantize(self, columns, x, up=None, **out):
        args = B.make_args(B.mega_moe_quantize_args, num_tokens=self.tokens, columns=columns, x_type=U.TYPE[x.dtype],
                           activation=B.MEGA_MOE_ACT_NONE if up is None else B.MEGA_MOE_ACT_SWIGLU, scale=B.MEGA_MOE_SCALE_ROW, x=x,
                           up=up, x_stride=x.stride(0), up_stride=0 if up is None else up.stride(0), **out)
        self._add(lambda s: B.mega_moe_quantize(args, s))

    def _heads(self, t):
        v = t.view(self.tokens, HQ + 2 * HK, DIM)
        return v[:, :HQ], v[:, HQ:HQ + HK], v[:, HQ + HK:]

    def _rotary(self):
        fields = dict(num_tokens=self.tokens, q_heads=HQ, k_heads=HK, head_dim=DIM, rotary_dim=DIM, layout=B.MEGA_MOE_ROTARY_HALF,
                      type=B.MEGA_MOE_BF16, weight_type=B.MEGA_MOE_F32, eps=EPS, q_weight=self.q_weight, k_weight=self.k_weight,
                      positions=self.positions, inv_freq=self.inv_freq)
        q, k, _ = self._heads(self.qkv)
        qo, ko, _ = self._heads(self.turned)
        strides = dict(q_stride=N, k_stride=N, q_out_stride=N, k_out_stride=N)
        args = B.make_args(B.mega_moe_rotary_args, q=q, k=k, q_out=qo, k_out=ko, **strides, **fields)
        self._add(lambda s: B.mega_moe_rotary(args, s))
        # gradients in place of a copy of their input, v's among them
        dq, dk, _ = self._heads(self.dqkv)
        self.d_rotary = B.make_args(B.mega_moe_rotary_backward_args, q=q, k=k, dq_out=dq, dk_out=dk, dq=dq, dk=dk, q_stride=N, k_stride=N,
                                    dq_out_stride=N, dk_out_stride=N, dq_stride=N, dk_stride=N, dq_weight=self.dq_weight,
                                    dk_weight=self.dk_weight, **fields)
        B.set_args(self.d_rotary, **U.workspace(B.mega_moe_rotary_workspace_bytes(self.d_rotary)))

    def _rotary_backward(self):
        self._add(lambda s: self.dqkv.copy_(self.dqkv_out))
        self._add(lambda s: B.mega_moe_rotary_backward(self.d_rotary, s))

    def run(self):
        s = U.current_stream()
        for step in self.steps:
            step(s)

    def named(self):
        return [(n, getattr(self, n)) for n in self.OUT] + [("dw " + k, v) for k, v in self.dw.items()]

    def clear(self):
        for _, t in self.named():
            t.zero_()

    def outputs(self):
        return {n: t.clone() for n, t in self.named()}

    def same(self, want, label):
        for n, t in self.named():
            assert torch.equal(t, want[n]), f"{label}: {n}"


@pytest.fixture(scope="module")
def eager():
    run = Run(1)
    run.run()
    torch.cuda.synchronize()
    assert run.layer.status() == 0
    yield run, run.outputs()
    run.layer.close()


def test_every_step_matches_the_reference(eager):
    run, o = eager
    w = run.w
    D.check_product(o["qkv"], o["q"], o["q_sf"], w["qkv"]["q"], w["qkv"]["q_sf"], "block", label="qkv")
    rotary = dict(positions=run.positions.cpu().numpy(), inv_freq=U.f64(run.inv_freq), eps=float(np.float32(EPS)))
    for i, weight in enumerate((run.q_weight, run.k_weight)):
        x, y = run._heads(o["qkv"])[i], run._heads(o["turned"])[i]
        want, mag = dense.rotary(U.f64(x), U.f64(weight), **rotary)
        U.near(y, want, mag, 40, f"heads {i}")
    D.check_product(o["gate_up"], o["q"], o["q_sf"], w["gate_up"]["q"], w["gate_up"]["q_sf"], "block", label="gate_up")
    gate, up = U.f64(o["gate_up"][:, :I]), U.f64(o["gate_up"][:, I:])
    h = dense.swiglu(gate, up)
    D.check_codes(o["a"], o["a_sf"], dense.rows_quotients(h), 16, "a")
    D.check_codes(o["at"], o["at_sf"], dense.transposed_quotients(h), 16, "at")
    inp = dict(x=o["q"].cpu().numpy(), x_sf=o["q_sf"].cpu().numpy(), topk_idx=run.idx.cpu().numpy(),
               topk_weights=run.weight.cpu().numpy(), **run.weights)
    G.check_y(o["routed"].view(torch.int16).cpu().numpy().view(np.uint16), moe.forward(inp)["y"], "routed")
    D.check_product(o["y"], o["a"], o["a_sf"], w["down"]["q"], w["down"]["q_sf"], "block", o["routed"], "y")
    D.check_codes(o["nt"], o["nt_sf"], dense.transposed_quotients(U.f64(o["n"])), 4, "nt")
    D.check_codes(o["dyq"], o["dyq_sf"], dense.rows_quotients(U.f64(run.dy)), 4, "dyq")
    D.check_codes(o["dyt"], o["dyt_sf"], dense.transposed_quotients(U.f64(run.dy)), 4, "dyt")
    D.check_product(o["da"], o["dyq"], o["dyq_sf"], w["down"]["qt"], w["down"]["qt_sf"], "block", label="da")
    D.check_product(o["dw down"], o["dyt"], o["dyt_sf"], o["at"], o["at_sf"], "row", run.before["down"], "dw down")
    dx, dx_mag, dup, dup_mag = dense.swiglu_backward(gate, up, U.f64(o["da"]))
    both, mag = np.concatenate([dx, dup], axis=1), np.concatenate([dx_mag, dup_mag], axis=1)
    D.check_codes(o["dgq"], o["dgq_sf"], dense.rows_quotients(both, mag), 16, "dgq")
    D.check_codes(o["dgt"], o["dgt_sf"], dense.transposed_quotients(both, mag), 16, "dgt")
    D.check_product(o["dn0"], o["dgq"], o["dgq_sf"], w["gate_up"]["qt"], w["gate_up"]["qt_sf"], "block", label="dn0")
    D.check_product(o["dw gate_up"], o["dgt"], o["dgt_sf"], o["nt"], o["nt_sf"], "row", run.before["gate_up"], "dw gate_up")
    for i, (weight, dw) in enumerate(((run.q_weight, "dq_weight"), (run.k_weight, "dk_weight"))):
        x, d, got = run._heads(o["qkv"])[i], run._heads(run.dqkv_out)[i], run._heads(o["dqkv"])[i]
        want, mag, dweight, dweight_mag = dense.rotary_backward(U.f64(x), U.f64(weight), U.f64(d), **rotary)
        U.near(got, want, mag, 96, f"dheads {i}")
        U.near(o[dw], dweight, dweight_mag, 96 + x.shape[0] * x.shape[1], dw)
    assert torch.equal(run._heads(o["dqkv"])[2], run._heads(run.dqkv_out)[2])
    D.check_codes(o["dpq"], o["dpq_sf"], dense.rows_quotients(U.f64(o["dqkv"])), 4, "dpq")
    D.check_product(o["dn"], o["dpq"], o["dpq_sf"], w["qkv"]["qt"], w["qkv"]["qt_sf"], "block", o["dn0"], "dn")
    D.check_product(o["dw qkv"], o["dpt"], o["dpt_sf"], o["nt"], o["nt_sf"], "row", run.before["qkv"], "dw qkv")


def test_run_repeats_bit_for_bit_also_on_another_stream(eager):
    run, o = eager
    for _ in range(3):
        run.clear()
        run.run()
        run.same(o, "again")
    side = torch.cuda.Stream()
    run.clear()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run.run()
    torch.cuda.current_stream().wait_stream(side)
    run.same(o, "side stream")


def _captured(run):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run.run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run.run()
    torch.cuda.synchronize()
    return graph


def test_captured_run_replays_to_the_eager_result(eager):
    run, o = eager
    graph = _captured(run)
    for i in range(4):
        run.clear()
        graph.replay()
        torch.cuda.synchronize()
        run.same(o, f"replay {i}")
        run.run()                                    # eager work between replays
        torch.cuda.synchronize()
        run.same(o, f"eager {i}")
    # new inputs in the same buffers
    before = run.h.clone()
    run.h.mul_(1.5)
    run.h[:, 0] = 100.0
    graph.replay()
    torch.cuda.synchronize()
    replayed = run.outputs()
    assert not torch.equal(replayed["y"], o["y"])
    run.run()
    run.same(replayed, "new inputs")
    run.h.copy_(before)
    run.run()
    run.same(o, "the old inputs again")


def test_two_captured_runs_at_once(eager):
    run, o = eager
    other = Run(2, tokens=300)                       # other tiles, with workspaces of their own
    try:
        other.run()
        torch.cuda.synchronize()
        want = other.outputs()
        graphs = [_captured(run), _captured(other)]
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(5):
            run.clear()
            other.clear()
            torch.cuda.synchronize()
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
            torch.cuda.synchronize()
            run.same(o, "first")
            other.same(want, "second")
    finally:
        other.layer.close()


def test_split_products_of_two_streams_at_once():
    # long sums split into parts: each call's partial sums are in its own workspace
    g = D.generator(4)
    calls = []
    for seed, (m, k, n) in enumerate([(136, 16384, 144), (264, 16384, 128)]):
        a, a_sf = D.operand(g, m, k)
        b, b_sf = D.operand(g, n, k)
        out = torch.zeros(m, n, device="cuda")
        args = D.product_args(a, a_sf, b, b_sf, out, "row")
        assert B.mega_moe_product_workspace_bytes(args) > 0
        calls.append((args, out, (a, a_sf, b, b_sf)))
    want = []
    for args, out, ops in calls:
        B.mega_moe_product(args, U.current_stream())
        D.check_product(out, *ops, "row")
        want.append(out.clone())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        for _, out, _ in calls:
            out.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for (args, _, _), s in zip(calls, streams):
                B.mega_moe_product(args, s.cuda_stream)
        torch.cuda.synchronize()
        for (_, out, _), w in zip(calls, want):
            assert torch.equal(out, w)
