"""The operators around the expert layer, measured: the norms on both sides of
it, the router's product and its selection, and the balance loss.

``listed()`` gives the named cases, ``draw(rng)`` more of the same ranges,
``prepare(case, seed)`` the inputs and output buffers of one on the GPU, and
``run(state)`` one pass.  With ``own`` false a pass computes the operator in
plain torch operations; with ``own`` true it calls the library.  ``work(case)``
is what a pass cannot do without, and ``exact(case, seed)`` the result from the
definition in float64.

Operators (T tokens, H hidden, E experts, k slots per token):

* ``norm``: r = residual_scale * h + gate * z with z = y or its RMS norm, and
  n = RMS norm of r, given as BF16 and as E4M3 codes with one scale per 128
  columns (what the expert layer takes).  ``norm_backward``: its gradients.
* ``logits``: x . w^T in float32.  ``logits_backward``: the gradients of x and w.
* ``topk``: the k best experts of every token, by softmax or sigmoid scores,
  with a selection bias and expert groups, and their weights.
* ``balance``: per-expert counts per sequence, the balance loss and the
  log-sum-exp (z) loss.
* ``router_backward``: the gradient of the logits from the top-k weights, from
  the losses, or from both.
"""

import math

import torch

own = False

EPS = 1e-6
RESIDUAL_SCALE = 0.875
BALANCE_COEFF = 1e-2
Z_COEFF = 1e-3
WEIGHT_SCALE = 2.5
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ---------------------------------------------------------------

def _norm(name, direction, tokens, hidden, stream, post, gate, quant):
    return {"name": name, "op": "norm" if direction == "forward" else "norm_backward", "tokens": tokens,
            "hidden": hidden, "stream": stream, "post": post, "gate": gate, "quant": quant}


def _logits(name, direction, tokens, hidden, experts, weight):
    return {"name": name, "op": "logits" if direction == "forward" else "logits_backward", "tokens": tokens,
            "hidden": hidden, "experts": experts, "weight": weight}


def _router(name, op, tokens, experts, topk, score, groups=1, bias=False, sequences=1, padded=False,
            parts="both", logits="f32"):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "topk": topk, "score": score,
            "groups": groups, "bias": bias, "sequences": sequences, "padded": padded, "parts": parts,
            "logits": logits}


def listed():
    return [
        # one new token in serving: the layer's output joins the residual stream, and the next block's input is made
        _norm("norm_1x7168", "forward", 1, 7168, "bf16", False, "none", True),
        # a prefill batch of a model that norms the block's output too and scales it per channel
        _norm("norm_8192x7168", "forward", 8192, 7168, "bf16", True, "channel", True),
        # a mid batch with the residual stream in float32 and a per-token gate; no codes are asked for
        _norm("norm_577x4096_f32", "forward", 577, 4096, "f32", False, "token", False),
        # a training step of the same block
        _norm("norm_backward_4096x4096", "backward", 4096, 4096, "bf16", True, "channel", False),
        # the router's product of a decode batch
        _logits("logits_128x7168x32", "forward", 128, 7168, 32, "bf16"),
        # of a prefill batch, with the router's weights kept in float32
        _logits("logits_8192x7168x256_f32", "forward", 8192, 7168, 256, "f32"),
        # a training step
        _logits("logits_backward_4096x4096x64", "backward", 4096, 4096, 64, "bf16"),
        # the selection of a decode batch
        _router("topk_128x32", "topk", 128, 32, 8, "softmax"),
        # of a prefill batch, over expert groups, with a selection bias
        _router("topk_8192x256_groups", "topk", 8192, 256, 8, "sigmoid", groups=8, bias=True),
        # the counts and losses of a mid batch
        _router("balance_576x32", "balance", 576, 32, 8, "softmax"),
        # of a training batch of packed sequences, with padding behind them
        _router("balance_8192x256_packed", "balance", 8192, 256, 8, "sigmoid", sequences=13, padded=True),
        # the gradient of that batch's logits, from the weights and the losses
        _router("router_backward_8192x256", "router_backward", 8192, 256, 8, "sigmoid", sequences=13, padded=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_backward", "logits", "logits_backward", "topk", "balance", "router_backward"])
    tokens = _log_int(rng, 1, 8192)
    if op in ("norm", "norm_backward"):
        hidden = 128 * _log_int(rng, 4, 64)
        tokens = min(tokens, 8192 * 7168 // hidden if op == "norm" else 4096 * 4096 // hidden)
        case = _norm("", "forward" if op == "norm" else "backward", tokens, hidden, rng.choice(["bf16", "f32"]),
                     rng.random() < 0.5, rng.choice(["none", "token", "channel", "full"]), op == "norm" and rng.random() < 0.5)
    elif op in ("logits", "logits_backward"):
        hidden = 128 * _log_int(rng, 4, 56)
        experts = _log_int(rng, 4, 512)
        most = 8192 * 7168 * 256 if op == "logits" else 4096 * 4096 * 64
        tokens = max(1, min(tokens, most // (hidden * experts)))
        case = _logits("", "forward" if op == "logits" else "backward", tokens, hidden, experts, rng.choice(["bf16", "f32"]))
    else:
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log_int(rng, 4, 512 // groups)
        tokens = max(1, min(tokens, 8192 * 256 // experts))
        # one renormalised weight is a constant: its gradient would be nothing but rounding
        topk = rng.randint(2 if op == "router_backward" else 1, min(8, experts // groups * max(1, groups // 2)))
        packed = rng.random() < 0.5
        case = _router("", op, tokens, experts, topk, rng.choice(["softmax", "sigmoid"]), groups if op == "topk" else 1,
                       rng.random() < 0.5, _log_int(rng, 1, max(1, min(tokens // 2, 64))) if packed else 1, packed and tokens > 8,
                       rng.choice(["weights", "losses", "both"]), rng.choice(["f32", "bf16"]))
    case.pop("name")
    return case


def _size(kind):
    return 2 if kind == "bf16" else 4


def work(case):
    op, T = case["op"], case["tokens"]
    if op in ("norm", "norm_backward"):
        H, s = case["hidden"], _size(case["stream"])
        gate = {"none": 0, "token": 4 * T, "channel": 4 * H, "full": 2 * T * H}[case["gate"]]
        if op == "norm":
            out = 2 * T * H + (T * H + T * H // 32 if case["quant"] else 0)
            return {"bytes": T * H * (2 * s + 2) + gate + out + 8 * H, "flops": 12 * T * H}
        return {"bytes": T * H * (3 * s + 6) + 2 * gate + 16 * H, "flops": 24 * T * H}
    E = case["experts"]
    if op in ("logits", "logits_backward"):
        H, s = case["hidden"], _size(case["weight"])
        if op == "logits":
            return {"bytes": 2 * T * H + s * E * H + 4 * T * E, "flops": 2 * T * H * E}
        return {"bytes": 4 * T * H + (s + 4) * E * H + 4 * T * E, "flops": 4 * T * H * E}
    k, s = case["topk"], _size(case["logits"])
    if op == "topk":
        return {"bytes": s * T * E + 8 * T * k, "flops": 8 * T * E}
    if op == "balance":
        return {"bytes": s * T * E + 4 * T * k + 8 * case["sequences"] * E, "flops": 8 * T * E}
    return {"bytes": (s + 4) * T * E + 8 * T * k, "flops": 16 * T * E}


# ---- what a program has in hand ----------------------------------------------

def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _outliers(v, g):
    """Activations with the few large channels that a residual stream has."""
    at = torch.randint(0, v.shape[1], (max(1, v.shape[1] // 1000),), generator=g, device="cuda")
    v[:, at] *= 50.0
    return v


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] in ("norm", "norm_backward"):
        _prepare_norm(s, case, g)
    elif case["op"] in ("logits", "logits_backward"):
        _prepare_logits(s, case, g)
    else:
        _prepare_router(s, case, g, seed)
    return s


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _prepare_norm(s, case, g):
    T, H, stream = case["tokens"], case["hidden"], DT[case["stream"]]
    gate = {"none": None, "token": (T,), "channel": (H,), "full": (T, H)}[case["gate"]]
    gate_type = torch.bfloat16 if case["gate"] == "full" else torch.float32
    s["y"] = _normal(g, T, H, scale=0.5, dtype=torch.bfloat16)
    s["gate"] = None if gate is None else torch.sigmoid(_normal(g, *gate)).to(gate_type)
    s["post"] = 1.0 + _normal(g, H, scale=0.1) if case["post"] else None
    s["pre"] = 1.0 + _normal(g, H, scale=0.1)
    stream_in = _outliers(_normal(g, T, H, scale=1.5), g).to(stream)
    if case["op"] == "norm":
        s["h"] = stream_in
        s["r"], s["n"] = _empty(T, H, dtype=stream), _empty(T, H, dtype=torch.bfloat16)
        s["q"] = _empty(T, H, dtype=torch.uint8) if case["quant"] else None
        s["q_sf"] = _empty(T, H // 128) if case["quant"] else None
        return
    s["r"] = stream_in
    s["dr"] = _normal(g, T, H, scale=1e-2, dtype=stream)
    s["dn"] = _normal(g, T, H, scale=1e-2, dtype=torch.bfloat16)
    s["dh"], s["dy"] = _empty(T, H, dtype=stream), _empty(T, H, dtype=torch.bfloat16)
    s["dgate"] = None if gate is None else _empty(*gate, dtype=gate_type)
    s["dpost"] = _empty(H) if case["post"] else None
    s["dpre"] = _empty(H)


def _prepare_logits(s, case, g):
    T, H, E = case["tokens"], case["hidden"], case["experts"]
    s["x"] = _outliers(_normal(g, T, H), g).to(torch.bfloat16)
    s["w"] = _normal(g, E, H, scale=0.02, dtype=DT[case["weight"]])
    s["logits"] = _empty(T, E)
    if case["op"] == "logits_backward":
        s["dlogits"] = _normal(g, T, E, scale=1e-3)
        s["dx"], s["dw"] = _empty(T, H, dtype=torch.bfloat16), _empty(E, H)


def _prepare_router(s, case, g, seed):
    T, E, k, B = case["tokens"], case["experts"], case["topk"], case["sequences"]
    # some experts are liked better than others, as in a trained router
    s["logits"] = (_normal(g, T, E) + 0.7 * _normal(g, E)).to(DT[case["logits"]])
    s["bias"] = _normal(g, E, scale=0.05) if case["bias"] else None
    used = T - T // 9 if case["padded"] else T
    cuts = torch.sort(torch.randperm(max(1, used - 1), generator=torch.Generator().manual_seed(seed))[:B - 1] + 1).values
    s["cu_seqlens"] = torch.cat([torch.zeros(1, dtype=torch.long), cuts, torch.tensor([used])]).to(torch.int32).cuda()
    s["token_mask"] = (torch.arange(T, device="cuda") < used).to(torch.uint8) if case["padded"] else None
    s["topk_idx"], s["topk_weights"] = _empty(T, k, dtype=torch.int32), _empty(T, k)
    if case["op"] == "topk":
        return
    s["topk_idx"].copy_(torch.topk(s["logits"].float(), k, dim=1).indices)
    if case["padded"]:
        s["topk_idx"][used:] = -1
    s["loss"], s["probs"] = _empty(2), _empty(B, E)
    s["counts"], s["tokens"] = _empty(B, E, dtype=torch.int32), _empty(B + 2, dtype=torch.int32)
    if case["op"] == "router_backward":
        s["counts"], s["tokens"] = _counts(s["topk_idx"], s["cu_seqlens"], s["token_mask"], T, E)
        s["dweights"] = _normal(g, T, k, scale=1e-3)
        s["dloss"] = 1.0 + _normal(g, 2, scale=0.1)
        s["dlogits"] = _empty(T, E)


# ---- one pass ------------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _rms(v):
    return v * torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS)


def _as_rows(case, gate):
    if gate is None:
        return 1.0
    return gate.float().unsqueeze(1) if case["gate"] == "token" else gate.float()


def _plain_norm(s):
    case, stream = s["case"], s["h"].dtype
    z = s["y"].float()
    if case["post"]:
        z = _rms(z) * s["post"]
    r = RESIDUAL_SCALE * s["h"].float() + _as_rows(case, s["gate"]) * z
    n = _rms(r) * s["pre"]
    out = {"r": r.to(stream), "n": n.to(torch.bfloat16)}
    if case["quant"]:
        T, H = n.shape
        blocks = n.view(T, H // 128, 128)
        sf = blocks.abs().amax(dim=2) / 448.0
        codes = torch.where(sf.unsqueeze(2) > 0, blocks / sf.unsqueeze(2), torch.zeros_like(blocks))
        out["q"], out["q_sf"] = codes.view(T, H).to(torch.float8_e4m3fn), sf
    return out


def _rms_grad(v, dout, weight):
    """The gradients of v and of weight for v * rsqrt(mean(v^2) + eps) * weight."""
    rs = torch.rsqrt(v.square().mean(dim=1, keepdim=True) + EPS)
    unit = v * rs
    u = dout if weight is None else dout * weight
    return rs * (u - unit * (u * unit).mean(dim=1, keepdim=True)), (dout * unit).sum(dim=0)


def _plain_norm_backward(s):
    case, stream = s["case"], s["r"].dtype
    dr, dpre = _rms_grad(s["r"].float(), s["dn"].float(), s["pre"])
    g = s["dr"].float() + dr
    out = {"dh": (RESIDUAL_SCALE * g).to(stream), "dpre": dpre}
    dz = _as_rows(case, s["gate"]) * g
    y = z = s["y"].float()
    dy = dz
    if case["post"]:
        z = _rms(y) * s["post"]
        dy, out["dpost"] = _rms_grad(y, dz, s["post"])
    out["dy"] = dy.to(torch.bfloat16)
    if s["gate"] is not None:
        dgate = z * g
        if case["gate"] != "full":
            dgate = dgate.sum(dim=1 if case["gate"] == "token" else 0)
        out["dgate"] = dgate.to(s["gate"].dtype)
    return out


def _plain_logits(s):
    return s["x"].float() @ s["w"].float().t()


def _plain_logits_backward(s):
    d = s["dlogits"]
    return {"dx": (d @ s["w"].float()).to(torch.bfloat16), "dw": d.t() @ s["x"].float()}


def _scores(case, l):
    return torch.softmax(l, dim=1) if case["score"] == "softmax" else torch.sigmoid(l)


def _plain_topk(s):
    case, E, k, G = s["case"], s["case"]["experts"], s["case"]["topk"], s["case"]["groups"]
    l = s["logits"].float()
    if s["bias"] is None and G == 1:
        choice = l.double()
    else:  # near ties decide which expert is taken: in 64 bits
        choice = _scores(case, l.double())
        if s["bias"] is not None:
            choice = choice + s["bias"].double()
    if G > 1:
        grouped = choice.view(-1, G, E // G)
        best = grouped.topk(min(2, E // G), dim=2).values.sum(dim=2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :_kept_groups(case)]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        choice = torch.where(keep.unsqueeze(2), grouped, -math.inf).view(-1, E)
    value, idx = torch.sort(choice, dim=1, descending=True, stable=True)
    value, idx = value[:, :k], idx[:, :k]
    live = value > -math.inf
    if s["token_mask"] is not None:
        live = live & (s["token_mask"] != 0).unsqueeze(1)
    w = torch.where(live, _scores(case, l).gather(1, idx), 0.0)
    total = w.sum(dim=1, keepdim=True)
    w = WEIGHT_SCALE * w / torch.where(total > 0, total, 1.0)
    return {"topk_idx": torch.where(live, idx, -1).to(torch.int32), "topk_weights": w}


def _kept_groups(case):
    return max(1, case["groups"] // 2)


def _sequence_rows(cu_seqlens, token_mask, T):
    """[B, T], 1 where a token is a valid one of a sequence."""
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    inside = (t >= cu_seqlens[:-1, None]) & (t < cu_seqlens[1:, None])
    if token_mask is not None:
        inside = inside & (token_mask != 0)
    return inside


def _counts(topk_idx, cu_seqlens, token_mask, T, E):
    """Routes per sequence and expert, and the valid tokens of each sequence, of all, and how many sequences have any."""
    rows = _sequence_rows(cu_seqlens, token_mask, T)
    picked = torch.zeros(T, E + 1, device="cuda").scatter_add_(
        1, torch.where(topk_idx < 0, E, topk_idx).long(), torch.ones_like(topk_idx, dtype=torch.float32))[:, :E]
    n = rows.sum(dim=1)
    tokens = torch.cat([n, n.sum().view(1), (n > 0).sum().view(1)])
    return (rows.float() @ picked).to(torch.int32), tokens.to(torch.int32)


def _probs(case, l):
    if case["score"] == "softmax":
        return torch.softmax(l, dim=1)
    p = torch.sigmoid(l)
    return p / p.sum(dim=1, keepdim=True)


def _plain_balance(s):
    case = s["case"]
    T, E, k = case["tokens"], case["experts"], case["topk"]
    l = s["logits"].float()
    counts, tokens = _counts(s["topk_idx"], s["cu_seqlens"], s["token_mask"], T, E)
    rows = _sequence_rows(s["cu_seqlens"], s["token_mask"], T)
    n = tokens[:-2].float().clamp(min=1.0)
    mean = (rows.float() @ _probs(case, l)) / n[:, None]
    share = counts.float() * (E / k) / n[:, None]
    balance = BALANCE_COEFF * (share * mean).sum() / tokens[-1].clamp(min=1)
    z = torch.where(rows.any(dim=0), torch.logsumexp(l, dim=1).square(), 0.0).sum() * Z_COEFF / tokens[-2].clamp(min=1)
    return {"loss": torch.stack([balance, z]), "counts": counts, "tokens": tokens, "probs": mean}


def _plain_router_backward(s):
    case = s["case"]
    T, E, k = case["tokens"], case["experts"], case["topk"]
    l = s["logits"].float()
    out = torch.zeros(T, E, device="cuda")
    live = s["topk_idx"] >= 0
    if s["token_mask"] is not None:
        live = live & (s["token_mask"] != 0).unsqueeze(1)
    at = torch.where(live, s["topk_idx"], 0).long()
    score = _scores(case, l)
    if case["parts"] != "losses":
        w = torch.where(live, score.gather(1, at), 0.0)
        total = w.sum(dim=1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        dw = torch.where(live, s["dweights"], 0.0)
        ds = torch.where(live, WEIGHT_SCALE / total * (dw - (dw * w).sum(dim=1, keepdim=True) / total), 0.0)
        ds = torch.zeros(T, E, device="cuda").scatter_add_(1, at, ds)
        if case["score"] == "sigmoid":
            out += ds * score * (1.0 - score)
        else:
            out += score * (ds - (ds * score).sum(dim=1, keepdim=True))
    if case["parts"] != "weights":
        rows = _sequence_rows(s["cu_seqlens"], s["token_mask"], T)
        n = s["tokens"][:-2].float().clamp(min=1.0)
        share = s["counts"].float() * (E / k) / n[:, None]
        scale = s["dloss"][0] * BALANCE_COEFF / (s["tokens"][-1].clamp(min=1) * n)
        f = rows.float().t() @ (share * scale[:, None])  # one row per token, 0 outside the sequences
        p = _probs(case, l)
        inner = f - (p * f).sum(dim=1, keepdim=True)
        if case["score"] == "sigmoid":
            out += inner * score * (1.0 - score) / score.sum(dim=1, keepdim=True)
        else:
            out += p * inner
        lse = torch.logsumexp(l, dim=1, keepdim=True) * (2.0 * Z_COEFF) * s["dloss"][1] / s["tokens"][-2].clamp(min=1)
        out += torch.where(rows.any(dim=0).unsqueeze(1), lse * torch.softmax(l, dim=1), 0.0)
    return out


_PLAIN = {"norm": _plain_norm, "norm_backward": _plain_norm_backward, "logits": _plain_logits,
          "logits_backward": _plain_logits_backward, "topk": _plain_topk, "balance": _plain_balance,
          "router_backward": _plain_router_backward}


# ---- the same through the library -----------------------------------------------

def _kept(s, make):
    """The argument block of a state's buffers, which a program fills in once and keeps."""
    if "args" not in s:
        from fp8_mixture_experts_amd import binding
        s["lib"] = binding
        s["args"] = make(binding)
    return s["lib"], s["args"], torch.cuda.current_stream().cuda_stream


def _workspace(s, nbytes):
    s["workspace"] = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
    return {"workspace": s["workspace"], "workspace_bytes": nbytes}


def _norm_types(B, s, stream):
    case = s["case"]
    kind = {"none": B.MEGA_MOE_GATE_NONE, "token": B.MEGA_MOE_GATE_TOKEN, "channel": B.MEGA_MOE_GATE_CHANNEL,
            "full": B.MEGA_MOE_GATE_FULL}[case["gate"]]
    return {"num_tokens": case["tokens"], "hidden": case["hidden"],
            "stream_type": B.MEGA_MOE_BF16 if stream == torch.bfloat16 else B.MEGA_MOE_F32,
            "weight_type": B.MEGA_MOE_F32, "gate_kind": kind,
            "gate_type": B.MEGA_MOE_BF16 if case["gate"] == "full" else B.MEGA_MOE_F32,
            "post_eps": EPS, "pre_eps": EPS, "residual_scale": RESIDUAL_SCALE,
            "y": s["y"], "gate": s["gate"], "post_weight": s["post"], "pre_weight": s["pre"]}


def _own_norm(s):
    B, args, stream = _kept(s, lambda B: B.make_args(
        B.mega_moe_norm_args, h=s["h"], r=s["r"], n=s["n"], q=s["q"], q_sf=s["q_sf"],
        **_norm_types(B, s, s["h"].dtype)))
    B.mega_moe_norm(args, stream)
    out = {"r": s["r"], "n": s["n"]}
    if s["q"] is not None:
        out["q"], out["q_sf"] = s["q"].view(torch.float8_e4m3fn), s["q_sf"]
    return out


def _own_norm_backward(s):
    def make(B):
        a = B.make_args(B.mega_moe_norm_backward_args, r=s["r"], dr=s["dr"], dn=s["dn"], dh=s["dh"], dy=s["dy"],
                        dgate=s["dgate"], dpost_weight=s["dpost"], dpre_weight=s["dpre"],
                        **_norm_types(B, s, s["r"].dtype))
        return B.set_args(a, **_workspace(s, B.mega_moe_norm_workspace_bytes(a)))
    B, args, stream = _kept(s, make)
    B.mega_moe_norm_backward(args, stream)
    out = {"dh": s["dh"], "dy": s["dy"], "dpre": s["dpre"]}
    if s["dpost"] is not None:
        out["dpost"] = s["dpost"]
    if s["dgate"] is not None:
        out["dgate"] = s["dgate"]
    return out


def _logits_args(B, s, **more):
    case = s["case"]
    a = B.make_args(B.mega_moe_router_logits_args, num_tokens=case["tokens"], hidden=case["hidden"],
                    num_experts=case["experts"],
                    weight_type=B.MEGA_MOE_BF16 if case["weight"] == "bf16" else B.MEGA_MOE_F32,
                    x=s["x"], w=s["w"], **more)
    return B.set_args(a, **_workspace(s, B.mega_moe_router_logits_workspace_bytes(a)))


def _own_logits(s):
    B, args, stream = _kept(s, lambda B: _logits_args(B, s, logits=s["logits"]))
    B.mega_moe_router_logits(args, stream)
    return s["logits"]


def _own_logits_backward(s):
    B, args, stream = _kept(s, lambda B: _logits_args(B, s, dlogits=s["dlogits"], dx=s["dx"], dw=s["dw"]))
    B.mega_moe_router_logits_backward(args, stream)
    return {"dx": s["dx"], "dw": s["dw"]}


def _score_types(B, s):
    case = s["case"]
    return {"num_tokens": case["tokens"], "num_experts": case["experts"], "num_topk": case["topk"],
            "logits_type": B.MEGA_MOE_F32 if case["logits"] == "f32" else B.MEGA_MOE_BF16,
            "score": B.MEGA_MOE_SCORE_SOFTMAX if case["score"] == "softmax" else B.MEGA_MOE_SCORE_SIGMOID,
            "logits": s["logits"], "token_mask": s["token_mask"]}


def _own_topk(s):
    case = s["case"]
    B, args, stream = _kept(s, lambda B: B.make_args(
        B.mega_moe_router_topk_args, renormalize=1, weight_scale=WEIGHT_SCALE, num_groups=case["groups"],
        topk_groups=_kept_groups(case), group_top=min(2, case["experts"] // case["groups"]), bias=s["bias"],
        topk_idx=s["topk_idx"], topk_weights=s["topk_weights"], **_score_types(B, s)))
    B.mega_moe_router_topk(args, stream)
    return {"topk_idx": s["topk_idx"], "topk_weights": s["topk_weights"]}


def _own_balance(s):
    def make(B):
        a = B.make_args(B.mega_moe_balance_loss_args, num_sequences=s["case"]["sequences"], cu_seqlens=s["cu_seqlens"],
                        topk_idx=s["topk_idx"], balance_coeff=BALANCE_COEFF, z_coeff=Z_COEFF, loss=s["loss"],
                        counts=s["counts"], tokens=s["tokens"], probs=s["probs"], **_score_types(B, s))
        return B.set_args(a, **_workspace(s, B.mega_moe_balance_loss_workspace_bytes(a)))
    B, args, stream = _kept(s, make)
    B.mega_moe_balance_loss(args, stream)
    return {"loss": s["loss"], "counts": s["counts"], "tokens": s["tokens"], "probs": s["probs"]}


def _own_router_backward(s):
    def make(B):
        parts = {}
        if s["case"]["parts"] != "losses":
            parts.update(dweights=s["dweights"], renormalize=1, weight_scale=WEIGHT_SCALE)
        if s["case"]["parts"] != "weights":
            parts.update(dloss=s["dloss"], num_sequences=s["case"]["sequences"], cu_seqlens=s["cu_seqlens"],
                         counts=s["counts"], tokens=s["tokens"], balance_coeff=BALANCE_COEFF, z_coeff=Z_COEFF)
        return B.make_args(B.mega_moe_router_backward_args, topk_idx=s["topk_idx"], dlogits=s["dlogits"],
                           **parts, **_score_types(B, s))
    B, args, stream = _kept(s, make)
    B.mega_moe_router_backward(args, stream)
    return s["dlogits"]


_OWN = {"norm": _own_norm, "norm_backward": _own_norm_backward, "logits": _own_logits,
        "logits_backward": _own_logits_backward, "topk": _own_topk, "balance": _own_balance,
        "router_backward": _own_router_backward}


# ---- the definitions in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return _EXACT[case["op"]](case, d)


def _gate64(case, d):
    """The gate of every element, [T, H]."""
    ones = torch.ones(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
    if case["gate"] == "none":
        return ones
    return torch.einsum("t,th->th", d["gate"], ones) if case["gate"] == "token" else d["gate"] * ones


def _length64(v):
    return torch.sqrt((v * v).sum(dim=1) / v.shape[1] + EPS)[:, None]


def _exact_norm(case, d):
    z = d["y"] / _length64(d["y"]) * d["post"] if case["post"] else d["y"]
    r = d["h"] * RESIDUAL_SCALE + z * _gate64(case, d)
    n = r / _length64(r) * d["pre"]
    out = {"r": r, "n": n}
    if case["quant"]:
        sf = n.reshape(-1, 128).abs().max(dim=1).values / 448.0
        out["q"] = (n.reshape(-1, 128) / sf[:, None]).reshape(n.shape)  # before it is rounded to a code
        out["q_sf"] = sf.reshape(n.shape[0], -1)
    return out


def _through_norm64(v, weight, dout):
    """dL/dv and dL/dweight: v / length(v) * weight, by the quotient rule."""
    length = _length64(v)
    dv = dout * weight / length
    dlength = -(dout * weight * v).sum(dim=1, keepdim=True) / length.square()
    return dv + dlength * v / (v.shape[1] * length), (dout * v / length).sum(dim=0)


def _exact_norm_backward(case, d):
    through, dpre = _through_norm64(d["r"], d["pre"], d["dn"])
    g = d["dr"] + through
    gate = _gate64(case, d)
    out = {"dh": g * RESIDUAL_SCALE, "dpre": dpre, "dy": g * gate}
    z = d["y"]
    if case["post"]:
        z = z / _length64(z) * d["post"]
        out["dy"], out["dpost"] = _through_norm64(d["y"], d["post"], g * gate)
    if case["gate"] != "none":
        how = {"token": "th,th->t", "channel": "th,th->h", "full": "th,th->th"}[case["gate"]]
        out["dgate"] = torch.einsum(how, z, g)
    return out


def _exact_logits(case, d):
    return torch.mm(d["x"], d["w"].t().contiguous())


def _exact_logits_backward(case, d):
    return {"dx": torch.mm(d["dlogits"], d["w"]), "dw": torch.mm(d["dlogits"].t().contiguous(), d["x"])}


def _score64(case, l):
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.max(dim=1, keepdim=True).values)
    return e / e.sum(dim=1, keepdim=True)


def _exact_topk(case, d):
    """The weights of the k best experts, one slot after another."""
    l = d["logits"]
    score = _score64(case, l)
    order = l.clone() if d["bias"] is None and case["groups"] == 1 else score.clone()
    if d["bias"] is not None:
        order += d["bias"]
    if case["groups"] > 1:
        size = case["experts"] // case["groups"]
        of_group = torch.stack([c.sort(dim=1).values[:, -2:].sum(dim=1) for c in order.split(size, dim=1)], dim=1)
        dropped = torch.ones_like(of_group, dtype=torch.bool)
        for _ in range(_kept_groups(case)):
            at = of_group.argmax(dim=1, keepdim=True)
            dropped.scatter_(1, at, False)
            of_group.scatter_(1, at, -math.inf)
        order[dropped.repeat_interleave(size, dim=1)] = -math.inf
    w = []
    for _ in range(case["topk"]):
        at = order.argmax(dim=1, keepdim=True)
        w.append(score.gather(1, at))
        order.scatter_(1, at, -math.inf)
    w = torch.cat(w, dim=1)
    w = WEIGHT_SCALE * w / w.sum(dim=1, keepdim=True)
    if d["token_mask"] is not None:
        w = w * (d["token_mask"] != 0)[:, None]
    return {"topk_idx": None, "topk_weights": w}


def _sequences(d):
    """The [first, last) tokens of every sequence; padding lies behind the last."""
    cu = d["cu_seqlens"].tolist()
    return list(zip(cu[:-1], cu[1:]))


def _shares64(case, d):
    """Each sequence's routes per expert over what an even spread would give."""
    share = []
    for lo, hi in _sequences(d):
        picked = d["topk_idx"][lo:hi].reshape(-1).long()
        share.append(torch.bincount(picked, minlength=case["experts"]).double() * case["experts"] / (case["topk"] * (hi - lo)))
    return share


def _exact_balance(case, d):
    l = d["logits"]
    p = _score64(case, l)
    p = p / p.sum(dim=1, keepdim=True)
    spans = _sequences(d)
    probs = torch.stack([p[lo:hi].mean(dim=0) for lo, hi in spans])
    balance = sum((f * m).sum() for f, m in zip(_shares64(case, d), probs)) * BALANCE_COEFF / len(spans)
    z = torch.log(torch.exp(l[:spans[-1][1]]).sum(dim=1)).square().mean() * Z_COEFF
    return {"loss": torch.stack([balance, z]), "counts": None, "tokens": None, "probs": probs}


def _exact_router_backward(case, d):
    """Row by row products with the Jacobian of the scores, sequence by sequence."""
    l = d["logits"]
    s = _score64(case, l)
    sig = case["score"] == "sigmoid"

    def through(ds):
        return ds * s * (1.0 - s) if sig else s * ds - s * (s * ds).sum(dim=1, keepdim=True)

    out = torch.zeros_like(l)
    spans = _sequences(d)
    end = spans[-1][1] if case["padded"] else case["tokens"]
    if case["parts"] != "losses":
        idx = d["topk_idx"][:end].long()
        w = s[:end].gather(1, idx)
        total = w.sum(dim=1, keepdim=True)
        dw = d["dweights"][:end]
        dsel = (dw * total - (dw * w).sum(dim=1, keepdim=True)) * WEIGHT_SCALE / total.square()
        ds = torch.zeros_like(l)
        ds[:end] = ds[:end].scatter(1, idx, dsel)
        out += through(ds)
    if case["parts"] != "weights":
        total = s.sum(dim=1, keepdim=True)
        df = torch.zeros_like(l)
        for (lo, hi), f in zip(spans, _shares64(case, d)):
            df[lo:hi] = f * d["dloss"][0] * BALANCE_COEFF / (len(spans) * (hi - lo))
        # p = s / sum(s): the quotient rule, then the scores' own
        out += through(df / total - (df * s).sum(dim=1, keepdim=True) / total.square())
        e = torch.exp(l)
        z = 2.0 * Z_COEFF * d["dloss"][1] / spans[-1][1] * torch.log(e.sum(dim=1, keepdim=True)) * e / e.sum(dim=1, keepdim=True)
        out[:spans[-1][1]] += z[:spans[-1][1]]
    return out


_EXACT = {"norm": _exact_norm, "norm_backward": _exact_norm_backward, "logits": _exact_logits,
          "logits_backward": _exact_logits_backward, "topk": _exact_topk, "balance": _exact_balance,
          "router_backward": _exact_router_backward}
