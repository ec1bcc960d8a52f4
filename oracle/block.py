"""Float64 reference of the operators around the layer (include/mega_moe.h).

Each function returns the values of the definition and, beside them, how much
of float32's rounding they can carry: ``*_mag`` arrays are sums of magnitudes
of the terms that an output is made of, so that an implementation in float32
is off by at most a small multiple of 2^-24 times them (plus the rounding of
the output's own type).  Nothing here is shared with the HIP sources.
"""

from __future__ import annotations

import numpy as np


def _inv_rms(v, eps):
    return 1.0 / np.sqrt(np.mean(v * v, axis=1, keepdims=True) + eps)


def _gate(kind, gate, T, H):
    if kind == "none":
        return np.ones((T, H))
    g = np.asarray(gate, np.float64)
    return np.broadcast_to(g[:, None] if kind == "token" else g, (T, H))


def norm(h, y=None, gate=None, kind="none", post=None, pre=None, scale=1.0, post_eps=0.0, pre_eps=0.0):
    h = np.asarray(h, np.float64)
    T, H = h.shape
    out = {}
    if y is None:
        r, r_mag = h, np.abs(h)
    else:
        z = np.asarray(y, np.float64)
        if post is not None:
            z = z * _inv_rms(z, post_eps) * post
        gz = _gate(kind, gate, T, H) * z
        r = scale * h + gz
        r_mag = np.abs(scale * h) + np.abs(gz)
    out["r"], out["r_mag"] = r, r_mag
    if pre is None:
        return out
    rs = _inv_rms(r, pre_eps)
    n = r * rs * pre
    out["n"], out["n_mag"] = n, np.abs(rs * pre) * r_mag + np.abs(n)
    if H % 128 == 0:
        sf = np.abs(n).reshape(T, H // 128, 128).max(axis=2) / 448.0
        wide = np.repeat(sf, 128, axis=1)
        out["q_sf"], out["q"] = sf, np.divide(n, wide, out=np.zeros_like(n), where=wide > 0)
        out["q_sf_mag"] = out["n_mag"].reshape(T, H // 128, 128).max(axis=2) / 448.0
    return out


def _norm_grad(v, weight, dout, dout_mag, eps):
    """Gradients of v * inv_rms(v) * weight, with the magnitudes."""
    rs = _inv_rms(v, eps)
    unit = v * rs
    u, um = dout * weight, dout_mag * np.abs(weight)
    dv = rs * (u - unit * np.mean(u * unit, axis=1, keepdims=True))
    dv_mag = rs * (um + np.abs(unit) * np.mean(um * np.abs(unit), axis=1, keepdims=True))
    return dv, dv_mag, (dout * unit).sum(axis=0), (dout_mag * np.abs(unit)).sum(axis=0)


def norm_backward(r, dr=None, dn=None, y=None, gate=None, kind="none", post=None, pre=None, scale=1.0,
                  post_eps=0.0, pre_eps=0.0):
    r = np.asarray(r, np.float64)
    T, H = r.shape
    out = {"dpre": np.zeros(H), "dpre_mag": np.zeros(H)}
    g = np.zeros((T, H)) if dr is None else np.asarray(dr, np.float64)
    g_mag = np.abs(g)
    if dn is not None:
        dn = np.asarray(dn, np.float64)
        d, dm, out["dpre"], out["dpre_mag"] = _norm_grad(r, pre, dn, np.abs(dn), pre_eps)
        g, g_mag = g + d, g_mag + dm
    out["dh"], out["dh_mag"] = scale * g, abs(scale) * g_mag
    if y is None:
        return out
    y = np.asarray(y, np.float64)
    G = _gate(kind, gate, T, H)
    z = y if post is None else y * _inv_rms(y, post_eps) * post
    dz, dz_mag = G * g, np.abs(G) * g_mag
    axis = {"token": 1, "channel": 0}.get(kind)
    out["dgate"], out["dgate_mag"] = z * g, np.abs(z) * g_mag
    if axis is not None:
        out["dgate"], out["dgate_mag"] = out["dgate"].sum(axis=axis), out["dgate_mag"].sum(axis=axis)
    if post is None:
        out["dy"], out["dy_mag"] = dz, dz_mag
    else:
        out["dy"], out["dy_mag"], out["dpost"], out["dpost_mag"] = _norm_grad(y, post, dz, dz_mag, post_eps)
    return out


def router_logits(x, w):
    x, w = np.asarray(x, np.float64), np.asarray(w, np.float64)
    return x @ w.T, np.abs(x) @ np.abs(w).T


def router_logits_backward(dlogits, x, w, dx_add=None):
    d, x, w = (np.asarray(v, np.float64) for v in (dlogits, x, w))
    dx, dx_mag = d @ w, np.abs(d) @ np.abs(w)
    if dx_add is not None:
        dx, dx_mag = dx + dx_add, dx_mag + np.abs(dx_add)
    return {"dx": dx, "dx_mag": dx_mag, "dw": d.T @ x, "dw_mag": np.abs(d).T @ np.abs(x)}


def _softmax(l):
    with np.errstate(invalid="ignore"):
        top = l.max(axis=1, keepdims=True)
        e = np.exp(l - np.where(np.isneginf(top), 0.0, top))
        total = e.sum(axis=1, keepdims=True)
        return np.divide(e, total, out=np.zeros_like(e), where=total != 0)


def _sigmoid(l):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-l))


def scores(l, score):
    return _softmax(l) if score == "softmax" else _sigmoid(l)


def router_topk(logits, k, score, bias=None, mask=None, renormalize=True, scale=1.0, groups=1, topk_groups=1,
                group_top=1):
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    s = scores(l, score)
    idx, wgt = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        c = l[t].copy() if bias is None and groups == 1 else s[t] + (0.0 if bias is None else np.asarray(bias, np.float64))
        c[~(l[t] > -np.inf) | ~(c > -np.inf)] = -np.inf
        if groups > 1:
            size = E // groups
            gs = [sum(sorted(c[g * size:(g + 1) * size])[-group_top:]) for g in range(groups)]
            kept = sorted(range(groups), key=lambda g: (-gs[g], g))[:topk_groups]
            for g in set(range(groups)) - set(kept):
                c[g * size:(g + 1) * size] = -np.inf
        order = [e for e in sorted(range(E), key=lambda e: (-c[e], e)) if c[e] > -np.inf][:k]
        idx[t, :len(order)] = order
        taken = s[t, order]
        total = taken.sum() if renormalize else 1.0
        wgt[t, :len(order)] = scale * taken / total if total else 0.0
    return idx, wgt


def _valid(T, cu, mask):
    """Each token's sequence, -1 outside of all or masked."""
    seq = np.full(T, -1)
    for b in range(len(cu) - 1):
        seq[cu[b]:cu[b + 1]] = b
    return seq if mask is None else np.where(np.asarray(mask) != 0, seq, -1)


def _lse(l):
    top = l.max(axis=1)
    with np.errstate(divide="ignore", invalid="ignore"):
        return np.where(np.isneginf(top), 0.0, top + np.log(np.exp(l - top[:, None]).sum(axis=1))), np.where(np.isneginf(top), 0.0, np.abs(top))


def probs(l, score):
    s = scores(l, score)
    total = s.sum(axis=1, keepdims=True)
    return np.divide(s, total, out=np.zeros_like(s), where=total != 0)


def balance_loss(logits, idx, score, cu=None, mask=None, balance_coeff=0.0, z_coeff=0.0):
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    k = idx.shape[1]
    cu = [0, T] if cu is None else list(cu)
    B = len(cu) - 1
    seq = _valid(T, cu, mask)
    p = probs(l, score)
    counts, mean, tokens = np.zeros((B, E), np.int64), np.zeros((B, E)), np.zeros(B + 2, np.int64)
    balance = 0.0
    for b in range(B):
        rows = seq == b
        n = int(rows.sum())
        tokens[b] = n
        if n == 0:
            continue
        picked = idx[rows].reshape(-1)
        counts[b] = np.bincount(picked[(picked >= 0) & (picked < E)], minlength=E)
        mean[b] = p[rows].sum(axis=0) / n
        balance += (E / (k * n)) * (counts[b] * mean[b]).sum()
    tokens[B], tokens[B + 1] = tokens[:B].sum(), (tokens[:B] > 0).sum()
    z = z_mag = 0.0
    if T:
        lse, top = _lse(l)
        live = seq >= 0
        z = (lse[live] ** 2).sum() / max(tokens[B], 1)
        z_mag = (np.abs(lse[live]) * (np.abs(lse[live]) + top[live] + 1.0)).sum() / max(tokens[B], 1)
    loss = np.array([balance_coeff * balance / max(tokens[B + 1], 1), z_coeff * z])
    return {"loss": loss, "loss_mag": np.abs([loss[0], z_coeff * z_mag]), "counts": counts, "tokens": tokens, "probs": mean}


def _through(l, s, score, ds, ds_mag):
    """ds through the scores: softmax's Jacobian, or the sigmoid's slope."""
    if score == "sigmoid":
        slope = s * _sigmoid(-l)
        return ds * slope, ds_mag * slope
    inner = (s * ds).sum(axis=1, keepdims=True)
    return s * (ds - inner), s * (ds_mag + (s * ds_mag).sum(axis=1, keepdims=True))


def router_backward(logits, score, idx=None, dweights=None, renormalize=True, scale=1.0, mask=None, dloss=None,
                    cu=None, counts=None, tokens=None, k=None, balance_coeff=0.0, z_coeff=0.0):
    l = np.asarray(logits, np.float64)
    T, E = l.shape
    s = scores(l, score)
    out, mag = np.zeros((T, E)), np.zeros((T, E))
    live = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    if dweights is not None:
        ds, dm = np.zeros((T, E)), np.zeros((T, E))
        for t in np.nonzero(live)[0]:
            slots = [j for j in range(idx.shape[1]) if 0 <= idx[t, j] < E]
            w = s[t, idx[t, slots]]
            dw = np.asarray(dweights, np.float64)[t, slots]
            total = w.sum()
            for j, e in enumerate(idx[t, slots]):
                if renormalize and total == 0:
                    continue
                f = scale / total if renormalize else scale
                mean = (dw * w).sum() / total if renormalize else 0.0
                mean_mag = (np.abs(dw) * w).sum() / total if renormalize else 0.0
                ds[t, e] += f * (dw[j] - mean)
                dm[t, e] += abs(f) * (abs(dw[j]) + mean_mag)
        d, m = _through(l, s, score, ds, dm)
        out, mag = out + d, mag + m
    if dloss is not None:
        cu = [0, T] if cu is None else list(cu)
        B = len(cu) - 1
        seq = _valid(T, cu, mask)
        rows = seq >= 0
        b = seq[rows]
        n = np.maximum(np.asarray(tokens[:B], np.float64), 1)
        f = np.zeros((T, E))
        f[rows] = (np.asarray(counts, np.float64) * (E / (k * n[:, None])) / n[:, None])[b]
        f *= dloss[0] * balance_coeff / max(int(tokens[B + 1]), 1)
        total = s.sum(axis=1, keepdims=True)
        total = np.where(total == 0, 1.0, total)
        inner = (s * f).sum(axis=1, keepdims=True) / total
        if score == "sigmoid":
            slope = s * _sigmoid(-l) / total
            out, mag = out + slope * (f - inner), mag + slope * (np.abs(f) + np.abs(inner))
        else:
            out, mag = out + s * (f - inner), mag + s * (np.abs(f) + np.abs(inner))
        lse, top = _lse(l)
        p = _softmax(l)
        c = 2.0 * z_coeff * dloss[1] / max(int(tokens[B]), 1)
        out[rows] += c * lse[rows, None] * p[rows]
        mag[rows] += abs(c) * (np.abs(lse[rows]) + top[rows] + 1.0)[:, None] * p[rows]
    out[~live], mag[~live] = 0.0, 0.0
    return out, mag
