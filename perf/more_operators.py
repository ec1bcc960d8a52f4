"""The dense path next to the expert layer, measured: the products of E4M3
operands, what makes their operands, and the head norms and the rotation behind
the projections of attention.

``listed()`` gives the named cases, ``draw(rng)`` more of the same ranges,
``prepare(case, seed)`` the inputs and output buffers of one on the GPU, and
``run(state)`` one pass.  With ``own`` false a pass computes the operator in
plain torch operations; with ``own`` true it calls the library.  ``work(case)``
is what a pass cannot do without, and ``exact(case, seed)`` the result from the
definition in float64.

Operators:

* ``product``: out = a . b^T (+ add) of E4M3 codes, a with one scale per row and
  128 columns, b with the same or one per 128 x 128 block; out in BF16 (a
  projection, the gradient of its input) or float32 (a weight's gradient).
* ``quantize``: x, or silu(x) * up, as codes and scales by rows, by columns (the
  transpose, padded to 128 tokens) or by 128 x 128 blocks, and in BF16.
* ``swiglu_backward``: the gradients of x and up, in BF16, as codes by rows, and
  by columns.
* ``rotary``: the RMS norm of every head of q and k, and the rotation of part of
  it by the token's position.  ``rotary_backward``: its gradients.
"""

import math

import torch

own = False

EPS = 1e-6
CLAMP = 7.0
ROTARY_SCALE = 1.2079441541679836      # 0.1 ln(8) + 1: contexts stretched eightfold
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- the cases ---------------------------------------------------------------

def _product(name, m, k, n, scale="block", out="bf16", add=False):
    return {"name": name, "op": "product", "m": m, "k": k, "n": n, "scale": scale, "out": out, "add": add}


def _quantize(name, tokens, columns, activation, kind="bf16", scale="row", h=False, codes=True, transposed=False, clamp=False):
    return {"name": name, "op": "quantize", "tokens": tokens, "columns": columns, "activation": activation, "kind": kind,
            "scale": scale, "h": h, "codes": codes, "transposed": transposed, "clamp": clamp}


def _swiglu(name, tokens, columns, kind="bf16", grads=True, codes=False, transposed=False, clamp=False):
    return {"name": name, "op": "swiglu_backward", "tokens": tokens, "columns": columns, "kind": kind, "grads": grads,
            "codes": codes, "transposed": transposed, "clamp": clamp}


def _rotary(name, direction, tokens, q_heads, k_heads, dim, rotary, start=0, layout="half", kind="bf16", weights=True,
            packed=True, far=0):
    return {"name": name, "op": "rotary" if direction == "forward" else "rotary_backward", "tokens": tokens, "q_heads": q_heads,
            "k_heads": k_heads, "dim": dim, "rotary": rotary, "start": start, "layout": layout, "kind": kind,
            "weights": weights, "packed": packed, "far": far}


def listed():
    return [
        # a projection for one new token in serving
        _product("product_1x7168x4096", 1, 7168, 4096),
        # the second product of a shared expert for a decode batch, added to the routed experts' output
        _product("product_128x2048x7168_add", 128, 2048, 7168, add=True),
        # a projection of a prefill batch
        _product("product_8192x7168x4096", 8192, 7168, 4096),
        # a weight's gradient in a training step: both operands have scales by rows, the sum over the tokens joins what earlier batches gave
        _product("product_4096x4001x2048_f32", 4096, 4001, 2048, scale="row", out="f32", add=True),
        # between the two products of a shared expert for a decode batch
        _quantize("quantize_128x2048_swiglu", 128, 2048, "swiglu"),
        # a training step keeps the codes of the transpose too, for the weight's gradient
        _quantize("quantize_8192x7168_both", 8192, 7168, "none", transposed=True),
        # the gradient between the two products, as both products behind it take it
        _swiglu("swiglu_backward_4096x2048_codes", 4096, 2048, grads=False, codes=True, transposed=True),
        # a ragged mid batch in BF16, with the values clamped
        _swiglu("swiglu_backward_577x2048", 577, 2048, clamp=True),
        # one new token far into a long context
        _rotary("rotary_1x64x8", "forward", 1, 64, 8, 128, 128, far=1000000),
        # a prefill batch, q and k lying in one projection's rows
        _rotary("rotary_8192x32x8", "forward", 8192, 32, 8, 128, 128),
        # a training step of the same heads
        _rotary("rotary_backward_4096x32x8", "backward", 4096, 32, 8, 128, 128),
        # a ragged batch in float32: the last 64 of 192 columns are rotated, in pairs of neighbours
        _rotary("rotary_backward_577x16x16_f32", "backward", 577, 16, 16, 192, 64, start=128, layout="interleaved", kind="f32"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["product", "product", "product", "quantize", "swiglu_backward", "rotary", "rotary_backward"])
    kind = rng.choice(["bf16", "bf16", "f32"])
    tokens = _log_int(rng, 1, 8192)
    if op == "product":
        out = rng.choice(["bf16", "bf16", "f32"])
        scale = rng.choice(["block", "row"])
        k, n = 128 * _log_int(rng, 1, 64), 8 * _log_int(rng, 8, 1024)
        if out == "f32":
            tokens, k, scale = 8 * _log_int(rng, 16, 512), _log_int(rng, 1, 8192), "row"
        tokens = max(1, min(tokens, 8192 * 7168 * 4096 // (k * n * (4 if out == "f32" else 1))))
        case = _product("", tokens, k, n, scale, out, rng.random() < 0.5)
    elif op == "quantize":
        columns = 128 * _log_int(rng, 1, 64)
        activation = rng.choice(["none", "swiglu"])
        tokens = max(1, min(tokens, 8192 * 7168 // (columns * (2 if activation == "swiglu" else 1) * (2 if kind == "f32" else 1))))
        which = rng.choice(["rows", "columns", "both", "values"])
        case = _quantize("", tokens, columns, activation, kind, rng.choice(["row", "row", "block"]), which == "values",
                         which != "columns", which in ("columns", "both"), rng.random() < 0.3 and activation == "swiglu")
    elif op == "swiglu_backward":
        columns = 128 * _log_int(rng, 1, 64)
        tokens = max(1, min(tokens, 4096 * 2048 // columns))
        which = rng.choice(["grads", "codes", "both", "all"])
        case = _swiglu("", tokens, columns, kind, which in ("grads", "all"), which != "grads", which in ("both", "all"),
                       rng.random() < 0.3)
    else:
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        rotary = rng.choice([dim // 16 * 16, dim // 2 // 16 * 16])
        q_heads, k_heads = rng.choice([(64, 8), (32, 8), (32, 4), (16, 16), (9, 3), (7, 1), (12, 0)])
        most = 8192 * 40 * 128 if op == "rotary" else 4096 * 40 * 128
        tokens = max(1, min(tokens, most // ((q_heads + k_heads) * dim * (2 if kind == "f32" else 1))))
        case = _rotary("", "forward" if op == "rotary" else "backward", tokens, q_heads, k_heads, dim, rotary,
                       rng.choice([0, (dim - rotary) // 8 * 8]), rng.choice(["half", "interleaved"]), kind, rng.random() < 0.7,
                       rng.random() < 0.7, rng.choice([0, _log_int(rng, 1, 1000000)]))
    case.pop("name")
    return case


def _size(kind):
    return 2 if kind == "bf16" else 4


def _up128(n):
    return (n + 127) // 128 * 128


def work(case):
    op = case["op"]
    if op == "product":
        m, k, n, s = case["m"], _up128(case["k"]), case["n"], _size(case["out"])
        b_scales = 4 * n * k // 128 if case["scale"] == "row" else 4 * _up128(n) * k // 16384
        return {"bytes": m * k + m * k // 32 + n * k + b_scales + (2 if case["add"] else 1) * s * m * n, "flops": 2 * m * k * n}
    if op in ("quantize", "swiglu_backward"):
        n, s = case["tokens"] * case["columns"], _size(case["kind"])
        codes = 1.0 if case.get("scale") == "block" else 1.0 + 1.0 / 32.0
        if op == "quantize":
            read = s * n * (2 if case["activation"] == "swiglu" else 1)
            return {"bytes": int(read + n * (2 * case["h"] + codes * (case["codes"] + case["transposed"]))), "flops": 10 * n}
        return {"bytes": int(3 * s * n + 2 * n * (s * case["grads"] + codes * (case["codes"] + case["transposed"]))), "flops": 20 * n}
    n, s = case["tokens"] * (case["q_heads"] + case["k_heads"]) * case["dim"], _size(case["kind"])
    if op == "rotary":
        return {"bytes": 2 * s * n, "flops": 10 * n}
    return {"bytes": (3 if case["weights"] else 2) * s * n, "flops": 20 * n}


# ---- what a program has in hand ----------------------------------------------

def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _outliers(v, g):
    """Activations with the few large channels that a residual stream has."""
    at = torch.randint(0, v.shape[1], (max(1, v.shape[1] // 1000),), generator=g, device="cuda")
    v[:, at] *= 20.0
    return v


def _empty(*shape, dtype=torch.float32):
    return torch.empty(shape, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    {"product": _prepare_product, "quantize": _prepare_quantize, "swiglu_backward": _prepare_swiglu,
     "rotary": _prepare_rotary, "rotary_backward": _prepare_rotary}[case["op"]](s, case, g)
    return s


def _stored(v, scale):
    """Codes and scales as a program has them stored: padded to whole blocks of columns."""
    rows, cols = v.shape
    v = torch.nn.functional.pad(v, (0, _up128(cols) - cols))
    if scale == "row":
        sf = v.abs().view(rows, -1, 128).amax(dim=2) / 448.0
        wide = sf.repeat_interleave(128, dim=1)
    else:
        p = torch.nn.functional.pad(v.abs(), (0, 0, 0, _up128(rows) - rows))
        sf = p.view(p.shape[0] // 128, 128, -1, 128).amax(dim=3).amax(dim=1) / 448.0
        wide = sf.repeat_interleave(128, dim=0)[:rows].repeat_interleave(128, dim=1)
    return torch.where(wide > 0, v / wide, 0.0).to(torch.float8_e4m3fn).view(torch.uint8), sf.contiguous()


def _prepare_product(s, case, g):
    m, k, n, out = case["m"], case["k"], case["n"], DT[case["out"]]
    if case["out"] == "f32":  # gradients of the output and activations, both transposed
        a, b = _normal(g, m, k, scale=1e-3), _outliers(_normal(g, k, n), g).t()
    else:
        a, b = _outliers(_normal(g, m, k), g), _normal(g, n, k, scale=0.02)
    s["a"], s["a_sf"] = _stored(a, "row")
    s["b"], s["b_sf"] = _stored(b.contiguous(), case["scale"])
    s["add"] = _normal(g, m, n, scale=0.1 if case["out"] == "f32" else 1.0, dtype=out) if case["add"] else None
    s["out"] = _empty(m, n, dtype=out)


def _prepare_quantize(s, case, g):
    T, C, kind = case["tokens"], case["columns"], DT[case["kind"]]
    swiglu = case["activation"] == "swiglu"
    both = _outliers(_normal(g, T, 2 * C if swiglu else C, scale=1.5), g).to(kind)  # gate and up are halves of one product's rows
    s["x"], s["up"] = (both[:, :C], both[:, C:]) if swiglu else (both, None)
    Tp, block = _up128(T), case["scale"] == "block"
    s["h"] = _empty(T, C, dtype=torch.bfloat16) if case["h"] else None
    s["q"] = _empty(T, C, dtype=torch.uint8) if case["codes"] else None
    s["q_sf"] = _empty(Tp // 128 if block else T, C // 128) if case["codes"] else None
    s["qt"] = _empty(C, Tp, dtype=torch.uint8) if case["transposed"] else None
    s["qt_sf"] = _empty(C // 128 if block else C, Tp // 128) if case["transposed"] else None


def _prepare_swiglu(s, case, g):
    T, C, kind = case["tokens"], case["columns"], DT[case["kind"]]
    both = _outliers(_normal(g, T, 2 * C, scale=1.5), g).to(kind)
    s["x"], s["up"] = both[:, :C], both[:, C:]
    s["dh"] = _normal(g, T, C, scale=1e-2, dtype=kind)
    Tp = _up128(T)
    s["dboth"] = _empty(T, 2 * C, dtype=kind) if case["grads"] else None
    s["q"] = _empty(T, 2 * C, dtype=torch.uint8) if case["codes"] else None
    s["q_sf"] = _empty(T, C // 64) if case["codes"] else None
    s["qt"] = _empty(2 * C, Tp, dtype=torch.uint8) if case["transposed"] else None
    s["qt_sf"] = _empty(2 * C, Tp // 128) if case["transposed"] else None


def _heads(s, case, name, make):
    """q and k [T, heads, D]: parts of one projection's rows (with the values behind them), or tensors of their own."""
    T, D, hq, hk = case["tokens"], case["dim"], case["q_heads"], case["k_heads"]
    if case["packed"]:
        whole = make(T, hq + 2 * hk, D)
        s[name[0]], s[name[1]] = whole[:, :hq], whole[:, hq:hq + hk]
    else:
        s[name[0]], s[name[1]] = make(T, hq, D), make(T, hk, D)
    if hk == 0:
        s[name[1]] = None


def _prepare_rotary(s, case, g):
    T, D, R, kind = case["tokens"], case["dim"], case["rotary"], DT[case["kind"]]
    _heads(s, case, ("q", "k"), lambda *shape: _normal(g, *shape, scale=1.5, dtype=kind))
    s["q_weight"] = 1.0 + _normal(g, D, scale=0.1) if case["weights"] else None
    s["k_weight"] = 1.0 + _normal(g, D, scale=0.1) if case["weights"] and case["k_heads"] else None
    # several prompts packed in one batch; or new tokens `far` into their context
    at = torch.arange(T, device="cuda")
    s["positions"] = (case["far"] + at if case["far"] else at % max(1, T * 2 // 3)).to(torch.int32)
    i = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    s["inv_freq"] = (10000.0 ** (-2.0 * i / max(R, 1)) / 8.0).to(torch.float32)
    heads = lambda *shape: _empty(*shape, dtype=kind)  # noqa: E731
    if case["op"] == "rotary":
        own_buffers = dict(case, packed=False)
        _heads(s, own_buffers, ("q_out", "k_out"), heads)
        return
    _heads(s, dict(case, packed=False), ("dq_out", "dk_out"), lambda *shape: _normal(g, *shape, scale=1e-2, dtype=kind))
    _heads(s, case, ("dq", "dk"), heads)
    s["dq_weight"] = _empty(D) if case["weights"] else None
    s["dk_weight"] = _empty(D) if s["k_weight"] is not None else None


# ---- one pass ------------------------------------------------------------------

def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


def _given(**outputs):
    return {name: v for name, v in outputs.items() if v is not None}


def _wide(sf, rows, scale):
    """A scale for every code."""
    if scale == "block":
        sf = sf.repeat_interleave(128, dim=0)[:rows]
    return sf.repeat_interleave(128, dim=1)


def _plain_product(s):
    case = s["case"]
    a = s["a"].view(torch.float8_e4m3fn).float() * _wide(s["a_sf"], case["m"], "row")
    b = s["b"].view(torch.float8_e4m3fn).float() * _wide(s["b_sf"], case["n"], case["scale"])
    out = a @ b.t()
    if s["add"] is not None:
        out = out + s["add"].float()
    return out.to(s["out"].dtype)


def _codes(v, block):
    """E4M3 codes and scales of v, by rows of 128 columns or by blocks."""
    rows, cols = v.shape
    if block:
        b = torch.nn.functional.pad(v, (0, 0, 0, _up128(rows) - rows)).view(-1, 128, cols // 128, 128)
        amax = b.abs().amax(dim=(1, 3), keepdim=True)
    else:
        b = v.reshape(rows, cols // 128, 128)
        amax = b.abs().amax(dim=2, keepdim=True)
    sf = amax / 448.0
    q = torch.where(sf > 0, b / torch.where(sf > 0, sf, 1.0), 0.0).to(torch.float8_e4m3fn)
    return q.reshape(-1, cols)[:rows], sf.reshape(-1, cols // 128)


def _all_codes(v, s, block):
    out = {}
    if s["q"] is not None:
        out["q"], out["q_sf"] = _codes(v, block)
    if s["qt"] is not None:
        vt = torch.nn.functional.pad(v, (0, 0, 0, _up128(v.shape[0]) - v.shape[0])).t()
        out["qt"], out["qt_sf"] = _codes(vt, block)
    return out


def _bounded(case, v):
    return v.clamp(-CLAMP, CLAMP) if case["clamp"] else v


def _plain_quantize(s):
    case = s["case"]
    v = s["x"].float()
    if case["activation"] == "swiglu":
        g = _bounded(case, v)
        v = g / (1.0 + torch.exp(-g)) * _bounded(case, s["up"].float())
    out = _all_codes(v, s, case["scale"] == "block")
    if s["h"] is not None:
        out["h"] = v.to(torch.bfloat16)
    return out


def _plain_swiglu_backward(s):
    case = s["case"]
    x, u, dh = s["x"].float(), s["up"].float(), s["dh"].float()
    g, ub = _bounded(case, x), _bounded(case, u)
    sig = 1.0 / (1.0 + torch.exp(-g))
    dx, du = dh * ub * sig * (1.0 + g * (1.0 - sig)), dh * g * sig
    if case["clamp"]:
        dx, du = torch.where(x.abs() > CLAMP, 0.0, dx), torch.where(u.abs() > CLAMP, 0.0, du)
    both = torch.cat([dx, du], dim=1)
    out = _all_codes(both, s, False)
    if case["grads"]:
        out["dboth"] = both.to(s["x"].dtype)
    return out


def _turns(s):
    """cos and sin of every token's angles, [T, 1, R/2]: in 64 bits, a position may be large."""
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    return torch.cos(angle).float() * ROTARY_SCALE, torch.sin(angle).float() * ROTARY_SCALE


def _pairs(case, v):
    """Both partners of every pair of the rotated part."""
    part = v[..., case["start"]:case["start"] + case["rotary"]]
    if case["layout"] == "half":
        return part[..., :case["rotary"] // 2], part[..., case["rotary"] // 2:]
    return part[..., 0::2], part[..., 1::2]


def _with_pairs(case, v, a, b):
    turned = torch.cat([a, b], dim=-1) if case["layout"] == "half" else torch.stack([a, b], dim=-1).flatten(-2)
    return torch.cat([v[..., :case["start"]], turned, v[..., case["start"] + case["rotary"]:]], dim=-1)


def _plain_rotary(s):
    case, out = s["case"], {}
    cos, sin = _turns(s)
    for name, x, w in (("q", s["q"], s["q_weight"]), ("k", s["k"], s["k_weight"])):
        if x is None:
            continue
        v = x.float()
        if w is not None:
            v = v * torch.rsqrt(v.square().mean(dim=-1, keepdim=True) + EPS) * w
        a, b = _pairs(case, v)
        out[name] = _with_pairs(case, v, a * cos - b * sin, b * cos + a * sin).to(x.dtype)
    return out


def _plain_rotary_backward(s):
    case, out = s["case"], {}
    cos, sin = _turns(s)
    for name, x, d, w in (("q", s["q"], s["dq_out"], s["q_weight"]), ("k", s["k"], s["dk_out"], s["k_weight"])):
        if x is None:
            continue
        u = d.float()
        a, b = _pairs(case, u)
        u = _with_pairs(case, u, a * cos + b * sin, b * cos - a * sin)
        if w is not None:
            v = x.float()
            rs = torch.rsqrt(v.square().mean(dim=-1, keepdim=True) + EPS)
            unit = v * rs
            out["d%s_weight" % name] = (u * unit).sum(dim=(0, 1))
            u = u * w
            u = rs * (u - unit * (u * unit).mean(dim=-1, keepdim=True))
        out["d" + name] = u.to(x.dtype)
    return out


_PLAIN = {"product": _plain_product, "quantize": _plain_quantize, "swiglu_backward": _plain_swiglu_backward,
          "rotary": _plain_rotary, "rotary_backward": _plain_rotary_backward}


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


def _type(B, kind):
    return B.MEGA_MOE_BF16 if kind == "bf16" else B.MEGA_MOE_F32


def _scale(B, scale):
    return B.MEGA_MOE_SCALE_BLOCK if scale == "block" else B.MEGA_MOE_SCALE_ROW


def _own_product(s):
    case = s["case"]

    def make(B):
        a = B.make_args(B.mega_moe_product_args, m=case["m"], n=case["n"], k=s["a"].shape[1], b_scale=_scale(B, case["scale"]),
                        out_type=_type(B, case["out"]), a=s["a"], a_sf=s["a_sf"], b=s["b"], b_sf=s["b_sf"], add=s["add"],
                        out=s["out"])
        return B.set_args(a, **_workspace(s, B.mega_moe_product_workspace_bytes(a)))
    B, args, stream = _kept(s, make)
    B.mega_moe_product(args, stream)
    return s["out"]


def _values(s):
    out = {}
    for q, sf in (("q", "q_sf"), ("qt", "qt_sf")):
        if s[q] is not None:
            out[q], out[sf] = s[q].view(torch.float8_e4m3fn), s[sf]
    return out


def _own_quantize(s):
    case = s["case"]
    B, args, stream = _kept(s, lambda B: B.make_args(
        B.mega_moe_quantize_args, num_tokens=case["tokens"], columns=case["columns"], x_type=_type(B, case["kind"]),
        activation=B.MEGA_MOE_ACT_SWIGLU if case["activation"] == "swiglu" else B.MEGA_MOE_ACT_NONE,
        scale=_scale(B, case["scale"]), activation_clamp=CLAMP if case["clamp"] else 0.0, x=s["x"], up=s["up"], h=s["h"],
        q=s["q"], q_sf=s["q_sf"], qt=s["qt"], qt_sf=s["qt_sf"], x_stride=s["x"].stride(0),
        up_stride=s["x"].stride(0) if s["up"] is not None else 0))
    B.mega_moe_quantize(args, stream)
    out = _values(s)
    if s["h"] is not None:
        out["h"] = s["h"]
    return out


def _own_swiglu_backward(s):
    case = s["case"]

    def make(B):
        grads = {}
        if case["grads"]:
            C = case["columns"]
            grads = {"dx": s["dboth"][:, :C], "dup": s["dboth"][:, C:], "dx_stride": 2 * C, "dup_stride": 2 * C}
        return B.make_args(B.mega_moe_swiglu_backward_args, num_tokens=case["tokens"], columns=case["columns"],
                           x_type=_type(B, case["kind"]), activation_clamp=CLAMP if case["clamp"] else 0.0, x=s["x"],
                           up=s["up"], dh=s["dh"], q=s["q"], q_sf=s["q_sf"], qt=s["qt"], qt_sf=s["qt_sf"],
                           x_stride=s["x"].stride(0), up_stride=s["up"].stride(0), **grads)
    B, args, stream = _kept(s, make)
    B.mega_moe_swiglu_backward(args, stream)
    return dict(_values(s), **_given(dboth=s["dboth"]))


def _rotary_types(B, s):
    case = s["case"]
    f = {"num_tokens": case["tokens"], "q_heads": case["q_heads"], "k_heads": case["k_heads"], "head_dim": case["dim"],
         "rotary_dim": case["rotary"], "rotary_start": case["start"],
         "layout": B.MEGA_MOE_ROTARY_HALF if case["layout"] == "half" else B.MEGA_MOE_ROTARY_INTERLEAVED,
         "type": _type(B, case["kind"]), "weight_type": B.MEGA_MOE_F32, "eps": EPS, "scale": ROTARY_SCALE,
         "q_weight": s["q_weight"], "k_weight": s["k_weight"], "positions": s["positions"], "inv_freq": s["inv_freq"]}
    for name in ("q", "k", "q_out", "k_out", "dq_out", "dk_out", "dq", "dk"):
        if s.get(name) is not None:
            f[name], f[name + "_stride"], f[name + "_head_stride"] = s[name], s[name].stride(0), s[name].stride(1)
    return f


def _own_rotary(s):
    B, args, stream = _kept(s, lambda B: B.make_args(B.mega_moe_rotary_args, **_rotary_types(B, s)))
    B.mega_moe_rotary(args, stream)
    return _given(q=s["q_out"], k=s["k_out"])


def _own_rotary_backward(s):
    def make(B):
        f = _rotary_types(B, s)
        a = B.make_args(B.mega_moe_rotary_backward_args, dq_weight=s["dq_weight"], dk_weight=s["dk_weight"], **f)
        return B.set_args(a, **_workspace(s, B.mega_moe_rotary_workspace_bytes(a)))
    B, args, stream = _kept(s, make)
    B.mega_moe_rotary_backward(args, stream)
    return _given(dq=s["dq"], dk=s["dk"], dq_weight=s["dq_weight"], dk_weight=s["dk_weight"])


_OWN = {"product": _own_product, "quantize": _own_quantize, "swiglu_backward": _own_swiglu_backward, "rotary": _own_rotary,
        "rotary_backward": _own_rotary_backward}


# ---- the definitions in 64 bits ----------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    return _EXACT[case["op"]](case, d)


def _exact_product(case, d):
    """One block of 128 after another: the codes' product, then both scales."""
    out = d["add"].clone() if case["add"] else torch.zeros(case["m"], case["n"], dtype=torch.float64, device="cuda")
    row = torch.arange(case["n"], device="cuda") // (128 if case["scale"] == "block" else 1)
    for i in range(d["a"].shape[1] // 128):
        at = slice(128 * i, 128 * i + 128)
        a, b = d["a"][:, at].contiguous().view(torch.float8_e4m3fn).double(), d["b"][:, at].contiguous().view(torch.float8_e4m3fn).double()
        out += torch.mm(a, b.t().contiguous()) * d["a_sf"][:, i, None] * d["b_sf"][row, i]
    return out


def _quotients64(h, names, d, block):
    """h over its scales, before it is rounded to codes."""
    out = {}
    for name, v in (("q", h), ("qt", h.t())):
        if d[name] is None:
            continue
        rows, cols = v.shape
        v = torch.cat([v, v.new_zeros(rows, _up128(cols) - cols)], dim=1)
        size = v.abs().reshape(rows, -1, 128).max(dim=2).values
        if block:
            size = torch.stack([c.max(dim=0).values for c in size.split(128)])
        sf = size / 448.0
        every = sf[torch.arange(rows, device="cuda") // (128 if block else 1)]
        out[name] = (v.reshape(rows, -1, 128) / every.clamp(min=1e-300)[:, :, None]).reshape(rows, -1)
        out[name + "_sf"] = sf
    return out


def _silu64(v):
    return v * torch.sigmoid(v)


def _exact_quantize(case, d):
    h = d["x"]
    if case["activation"] == "swiglu":
        most = CLAMP if case["clamp"] else math.inf
        h = _silu64(torch.clip(d["x"], -most, most)) * torch.clip(d["up"], -most, most)
    out = _quotients64(h, ("q", "qt"), d, case["scale"] == "block")
    if case["h"]:
        out["h"] = h
    return out


def _exact_swiglu_backward(case, d):
    most = CLAMP if case["clamp"] else math.inf
    x, u = torch.clip(d["x"], -most, most), torch.clip(d["up"], -most, most)
    e = torch.exp(-x.abs())
    s = torch.where(x < 0, e, 1.0) / (1.0 + e)
    slope = s + x * e / (1.0 + e).square()
    both = torch.cat([d["dh"] * u * slope * (x == d["x"]), d["dh"] * _silu64(x) * (u == d["up"])], dim=1)
    out = _quotients64(both, ("q", "qt"), d, False)
    if case["grads"]:
        out["dboth"] = both
    return out


def _turn64(case, d, v, back):
    """The rotated part as complex numbers times e^(i angle)."""
    T, heads, lo, R = v.shape[0], v.shape[1], case["start"], case["rotary"]
    part = v[..., lo:lo + R]
    if case["layout"] == "half":
        part = part.reshape(T, heads, 2, R // 2).transpose(2, 3)
    z = torch.view_as_complex(part.reshape(T, heads, R // 2, 2).contiguous())
    angle = torch.outer(d["positions"].double(), d["inv_freq"])[:, None]
    z = z * torch.polar(torch.full_like(angle, ROTARY_SCALE), -angle if back else angle)
    part = torch.view_as_real(z)
    if case["layout"] == "half":
        part = part.transpose(2, 3)
    out = v.clone()
    out[..., lo:lo + R] = part.reshape(T, heads, R)
    return out


def _length64(v):
    return torch.sqrt((v * v).sum(dim=-1, keepdim=True) / v.shape[-1] + EPS)


def _exact_rotary(case, d):
    out = {}
    for name in ("q", "k"):
        v, w = d[name], d[name + "_weight"]
        if v is not None:
            out[name] = _turn64(case, d, v if w is None else v / _length64(v) * w, False)
    return out


def _exact_rotary_backward(case, d):
    """Through the rotation, then v / length(v) * w by the quotient rule."""
    out = {}
    for name in ("q", "k"):
        v, w = d[name], d[name + "_weight"]
        if v is None:
            continue
        u = _turn64(case, d, d["d%s_out" % name], True)
        if w is not None:
            n = _length64(v)
            out["d%s_weight" % name] = torch.mm(torch.ones(1, v.shape[0] * v.shape[1], dtype=torch.float64, device="cuda"),
                                                (u * v / n).reshape(-1, case["dim"]))[0]
            u = u * w
            u = u / n - v * (u * v).sum(dim=-1, keepdim=True) / (case["dim"] * n ** 3)
        out["d" + name] = u
    return out


_EXACT = {"product": _exact_product, "quantize": _exact_quantize, "swiglu_backward": _exact_swiglu_backward,
          "rotary": _exact_rotary, "rotary_backward": _exact_rotary_backward}
