"""The operators around the layer in a run, as a model's block uses them: the
norm that makes the layer's input, the router's product and selection, the
layer, and the norm that takes its output back into the residual stream; and
the gradients of the router behind it.  Each step is checked against the
float64 reference on the values that the step before it gave; then the whole
run eagerly again, on another stream, from a captured graph with eager work
between its replays, and two captured runs at once.
"""

import numpy as np
import pytest
import torch

from fp8_mixture_experts_amd import binding as B
from fp8_mixture_experts_amd import synthetic as S
from oracle import block, codecs, moe
from tests import block_util as U
from tests import gpu_util as G

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
T, H, I, E, K = 61, 512, 256, 24, 4
GROUPS, KEPT = 4, 2


class Run:
    """One block's buffers, argument blocks and layer handle."""

    def __init__(self, seed, tokens=T):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s, dtype=F32, scale=1.0: (torch.randn(*s, generator=g, device="cuda") * scale).to(dtype)   # noqa: E731
        self.tokens = tokens
        self.weights = S.make_weights(S.custom(tokens=tokens, hidden=H, intermediate=I, experts=E, topk=K, weight_seed=5))
        self.dev = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in self.weights.items()}
        self.h, self.pre, self.next_pre = r(tokens, H, dtype=BF16), 1 + r(H, scale=0.1), 1 + r(H, scale=0.1)
        self.post, self.gate = 1 + r(H, scale=0.1), r(H)
        self.w, self.bias = r(E, H, scale=0.05), r(E, scale=0.02)
        self.dn, self.dweights, self.dloss = r(tokens, H, dtype=BF16, scale=0.01), r(tokens, K), 1 + r(2, scale=0.1)
        new = lambda *s, dtype=F32: torch.zeros(s, dtype=dtype, device="cuda")   # noqa: E731
        self.n, self.q, self.q_sf = new(tokens, H, dtype=BF16), new(tokens, H, dtype=torch.uint8), new(tokens, H // 128)
        self.logits, self.idx, self.weight = new(tokens, E), new(tokens, K, dtype=torch.int32), new(tokens, K)
        self.y, self.r, self.next_n = new(tokens, H, dtype=BF16), new(tokens, H, dtype=BF16), new(tokens, H, dtype=BF16)
        self.loss, self.counts, self.valid, self.probs = new(2), new(1, E, dtype=torch.int32), new(3, dtype=torch.int32), new(1, E)
        self.dlogits, self.dx, self.dw = new(tokens, E), new(tokens, H, dtype=BF16), new(E, H)
        self.dh, self.dpre = new(tokens, H, dtype=BF16), new(H)
        self.layer = B.MegaMoE(E, H, I, K, tokens)
        norm = dict(num_tokens=tokens, hidden=H, weight_type=B.MEGA_MOE_F32, gate_type=B.MEGA_MOE_F32, pre_eps=1e-6, post_eps=1e-6)
        route = dict(num_tokens=tokens, num_experts=E, num_topk=K, logits_type=B.MEGA_MOE_F32, score=B.MEGA_MOE_SCORE_SIGMOID,
                     logits=self.logits, topk_idx=self.idx)
        self.a_norm = B.make_args(B.mega_moe_norm_args, residual_scale=1.0, h=self.h, pre_weight=self.pre, n=self.n, q=self.q,
                                  q_sf=self.q_sf, **norm)
        self.a_logits = B.make_args(B.mega_moe_router_logits_args, num_tokens=tokens, hidden=H, num_experts=E,
                                    weight_type=B.MEGA_MOE_F32, x=self.n, w=self.w, logits=self.logits, dlogits=self.dlogits,
                                    dx=self.dx, dx_add=self.dn, dw=self.dw)
        B.set_args(self.a_logits, **U.workspace(B.mega_moe_router_logits_workspace_bytes(self.a_logits)))
        self.a_topk = B.make_args(B.mega_moe_router_topk_args, renormalize=1, weight_scale=2.0, num_groups=GROUPS,
                                  topk_groups=KEPT, group_top=2, bias=self.bias, topk_weights=self.weight, **route)
        self.a_next = B.make_args(B.mega_moe_norm_args, residual_scale=0.9, h=self.h, y=self.y, post_weight=self.post,
                                  gate_kind=B.MEGA_MOE_GATE_CHANNEL, gate=self.gate, pre_weight=self.next_pre, r=self.r,
                                  n=self.next_n, **norm)
        self.a_loss = B.make_args(B.mega_moe_balance_loss_args, balance_coeff=0.01, z_coeff=0.001, loss=self.loss,
                                  counts=self.counts, tokens=self.valid, probs=self.probs, **route)
        B.set_args(self.a_loss, **U.workspace(B.mega_moe_balance_loss_workspace_bytes(self.a_loss)))
        self.a_dlogits = B.make_args(B.mega_moe_router_backward_args, renormalize=1, weight_scale=2.0, balance_coeff=0.01,
                                     z_coeff=0.001, dweights=self.dweights, dloss=self.dloss, counts=self.counts,
                                     tokens=self.valid, dlogits=self.dlogits, **route)
        self.a_dnorm = B.make_args(B.mega_moe_norm_backward_args, residual_scale=1.0, r=self.h, dn=self.dx, pre_weight=self.pre,
                                   dh=self.dh, dpre_weight=self.dpre, **norm)
        B.set_args(self.a_dnorm, **U.workspace(B.mega_moe_norm_workspace_bytes(self.a_dnorm)))

    OUT = ("n", "q", "q_sf", "logits", "idx", "weight", "y", "r", "next_n", "loss", "counts", "valid", "probs", "dlogits", "dx",
           "dw", "dh", "dpre")

    def run(self):
        s, d = U.current_stream(), self.dev
        B.mega_moe_norm(self.a_norm, s)
        B.mega_moe_router_logits(self.a_logits, s)
        B.mega_moe_router_topk(self.a_topk, s)
        B.mega_moe_forward(self.layer.handle, self.tokens, self.q, self.q_sf, self.idx, self.weight, d["w1"], d["w1_sf"],
                           d["w2"], d["w2_sf"], self.y, s)
        B.mega_moe_norm(self.a_next, s)
        B.mega_moe_balance_loss(self.a_loss, s)
        B.mega_moe_router_backward(self.a_dlogits, s)
        B.mega_moe_router_logits_backward(self.a_logits, s)
        B.mega_moe_norm_backward(self.a_dnorm, s)

    def clear(self):
        for name in self.OUT:
            getattr(self, name).zero_()

    def outputs(self):
        return {name: getattr(self, name).clone() for name in self.OUT}

    def same(self, want, label):
        for name in self.OUT:
            assert torch.equal(getattr(self, name), want[name]), f"{label}: {name}"


@pytest.fixture(scope="module")
def eager():
    run = Run(1)
    run.run()
    torch.cuda.synchronize()
    assert run.layer.status() == 0
    yield run, run.outputs()
    run.layer.close()


def _np(t):
    return t.cpu().numpy()


def test_every_step_matches_the_reference(eager):
    run, o = eager
    n = block.norm(U.f64(run.h), pre=U.f64(run.pre), pre_eps=1e-6)
    U.near(o["n"], n["n"], n["n_mag"], 48, "n")
    U.near(o["q_sf"], n["q_sf"], n["q_sf_mag"], 48, "q_sf")
    logits, mag = block.router_logits(U.f64(o["n"]), U.f64(run.w))
    U.near(o["logits"], logits, mag, H + 16, "logits")
    idx, weight = block.router_topk(U.f64(o["logits"]), K, "sigmoid", U.f64(run.bias), None, True, 2.0, GROUPS, KEPT, 2)
    assert np.array_equal(_np(o["idx"]), idx)
    U.near(o["weight"], weight, weight, 48, "weight")
    inp = dict(x=_np(o["q"]), x_sf=_np(o["q_sf"]), topk_idx=_np(o["idx"]), topk_weights=_np(o["weight"]), **run.weights)
    G.check_y(_np(o["y"].view(torch.int16)).view(np.uint16), moe.forward(inp)["y"], "y")
    # residual_scale and the epsilons are float32 in the call
    nx = block.norm(U.f64(run.h), U.f64(o["y"]), U.f64(run.gate), "channel", U.f64(run.post), U.f64(run.next_pre),
                    float(np.float32(0.9)), float(np.float32(1e-6)), float(np.float32(1e-6)))
    U.near(o["r"], nx["r"], nx["r_mag"], 48, "r")
    U.near(o["next_n"], nx["n"], nx["n_mag"], 48, "next_n")
    coeff = float(np.float32(0.01)), float(np.float32(0.001))
    bal = block.balance_loss(U.f64(o["logits"]), idx, "sigmoid", None, None, *coeff)
    assert np.array_equal(_np(o["counts"]), bal["counts"]) and np.array_equal(_np(o["valid"]), bal["tokens"])
    U.near(o["loss"], bal["loss"], bal["loss_mag"], 128 + T, "loss")
    dl, mag = block.router_backward(U.f64(o["logits"]), "sigmoid", idx, U.f64(run.dweights), True, 2.0, None, U.f64(run.dloss),
                                    None, bal["counts"], bal["tokens"], K, *coeff)
    U.near(o["dlogits"], dl, mag, 128, "dlogits")
    g = block.router_logits_backward(U.f64(o["dlogits"]), U.f64(o["n"]), U.f64(run.w), U.f64(run.dn))
    U.near(o["dx"], g["dx"], g["dx_mag"], 512 + E + 16, "dx")
    U.near(o["dw"], g["dw"], g["dw_mag"], T + 16, "dw")
    d = block.norm_backward(U.f64(run.h), dn=U.f64(o["dx"]), pre=U.f64(run.pre), pre_eps=float(np.float32(1e-6)))
    U.near(o["dh"], d["dh"], d["dh_mag"], 96, "dh")
    U.near(o["dpre"], d["dpre"], d["dpre_mag"], 96 + T, "dpre")


def test_router_gradient_matches_differences(eager):
    # along one direction, through the library's own forward calls
    run, o = eager
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    v = torch.randn(T, E, generator=g, device="cuda")

    def value(step):
        run.logits.copy_(o["logits"] + step * v)
        run.idx.copy_(o["idx"])
        B.mega_moe_balance_loss(run.a_loss, U.current_stream())
        s = torch.sigmoid(run.logits.double()).gather(1, o["idx"].long())
        w = 2.0 * s / s.sum(dim=1, keepdim=True)
        return float((w * run.dweights.double()).sum() + (run.loss.double() * run.dloss.double()).sum())

    step = 1e-3
    got = (value(step) - value(-step)) / (2 * step)
    want = float((o["dlogits"].double() * v.double()).sum())
    # truncation step^2 of a third derivative of the order of the sum of |v|^3
    # |dweights|, and the losses' float32 rounding over the step
    slack = step ** 2 * float((v.abs() ** 3).sum()) + 1e-5
    assert abs(got - want) <= slack, (got, want, slack)
    run.run()


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
    graph.replay()
    torch.cuda.synchronize()
    replayed = run.outputs()
    run.run()
    run.same(replayed, "new inputs")
    run.h.copy_(before)
    run.run()
    run.same(o, "the old inputs again")


def test_two_captured_runs_at_once(eager):
    run, o = eager
    other = Run(2, tokens=300)                       # the large batch's kernels, with workspaces of their own
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
