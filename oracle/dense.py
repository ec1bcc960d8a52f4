"""Float64 reference of the dense path next to the layer (include/mega_moe.h):
products of E4M3 operands, what makes them, head norms with rotation.

As in ``oracle/block.py``, ``*_mag`` arrays are sums of magnitudes of the terms
that an output is made of: a float32 implementation is off by at most a small
multiple of 2^-24 times them.  Nothing here is shared with the HIP sources.
"""

from __future__ import annotations

import math

import numpy as np

BLOCK = 128


def _blocks(n):
    return -(-n // BLOCK)


def wide_scales(sf, rows, by_rows):
    """One scale per code of a [rows, k] operand."""
    sf = np.asarray(sf, np.float64)
    if not by_rows:
        sf = np.repeat(sf, BLOCK, axis=0)[:rows]
    return np.repeat(sf, BLOCK, axis=1)


def product(a, a_sf, b, b_sf, b_by_rows, add=None):
    """out = a . b^T + add; a and b are the codes' values.  ``mag`` is the sum of
    magnitudes, ``cut`` what the FP8 matrix instruction may leave out of it: up to
    2^-16 of a group's largest product for each of its 64 products."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    m, k = a.shape
    n = b.shape[0]
    wa, wb = wide_scales(a_sf, m, True), wide_scales(b_sf, n, b_by_rows)
    out = (a * wa) @ (b * wb).T
    mag = (np.abs(a) * np.abs(wa)) @ (np.abs(b) * np.abs(wb)).T
    cut = np.zeros((m, n))
    for s in range(0, k, 64):
        # the largest product of a group is at most the product of the largest codes
        cut += 64 * 2.0 ** -16 * np.outer(np.abs((a * wa)[:, s:s + 64]).max(axis=1), np.abs((b * wb)[:, s:s + 64]).max(axis=1))
    if add is not None:
        add = np.asarray(add, np.float64)
        out, mag = out + add, mag + np.abs(add)
    return out, mag, cut


def rows_quotients(v, v_mag=None):
    """sf [rows, cols / 128] and v / sf before it is rounded to codes, by rows of 128."""
    rows, cols = v.shape
    sf = np.abs(v).reshape(rows, -1, BLOCK).max(axis=2) / 448.0
    wide = np.repeat(sf, BLOCK, axis=1)
    q = np.divide(v, wide, out=np.zeros_like(v), where=wide > 0)
    mag = np.abs(v) if v_mag is None else v_mag
    return {"sf": sf, "q": q, "sf_mag": mag.reshape(rows, -1, BLOCK).max(axis=2) / 448.0,
            "q_mag": np.divide(mag, wide, out=np.zeros_like(v), where=wide > 0)}


def _padded(v):
    return np.concatenate([v, np.zeros((_blocks(v.shape[0]) * BLOCK - v.shape[0], v.shape[1]))])


def transposed_quotients(v, v_mag=None):
    return rows_quotients(_padded(v).T.copy(), None if v_mag is None else _padded(v_mag).T.copy())


def block_quotients(v):
    """By blocks of 128 x 128: sf [rows / 128, cols / 128] and the quotients."""
    p = _padded(v)
    sf = np.abs(p).reshape(p.shape[0] // BLOCK, BLOCK, -1, BLOCK).max(axis=(1, 3)) / 448.0
    wide = wide_scales(sf, v.shape[0], False)
    return {"sf": sf, "q": np.divide(v, wide, out=np.zeros_like(v), where=wide > 0)}


def _sigmoid(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0, e) / (1.0 + e)


def swiglu(x, up, clamp=0.0):
    c = clamp or np.inf
    g, u = np.clip(np.asarray(x, np.float64), -c, c), np.clip(np.asarray(up, np.float64), -c, c)
    return g * _sigmoid(g) * u


def swiglu_backward(x, up, dh, clamp=0.0):
    """dx and dup, with the magnitudes of their terms."""
    c = clamp or np.inf
    x, up, dh = (np.asarray(v, np.float64) for v in (x, up, dh))
    g, u = np.clip(x, -c, c), np.clip(up, -c, c)
    s = _sigmoid(g)
    dx, dx_mag = dh * u * s * (1.0 + g * (1.0 - s)), np.abs(dh * u) * s * (1.0 + np.abs(g) * (1.0 - s))
    dup = dh * g * s
    inside_x, inside_u = np.abs(x) <= c, np.abs(up) <= c
    return dx * inside_x, dx_mag * inside_x, dup * inside_u, np.abs(dup) * inside_u


def _turned(v, mag, positions, inv_freq, start, interleaved, scale, sign):
    """v [T, heads, D] with its rotated part turned by sign * angle."""
    half = len(inv_freq)
    out, out_mag = v.copy(), mag.copy()
    at = start + (2 * np.arange(half) if interleaved else np.arange(half))
    other = at + (1 if interleaved else half)
    angle = np.asarray(positions, np.float64)[:, None, None] * np.asarray(inv_freq, np.float64)
    c, s = np.cos(angle) * scale, np.sin(angle) * scale * sign
    a, b = v[..., at], v[..., other]
    out[..., at], out[..., other] = a * c - b * s, b * c + a * s
    am, bm = mag[..., at], mag[..., other]
    # cos and sin carry an absolute error in units of float32's rounding
    out_mag[..., at] = out_mag[..., other] = (am + bm) * abs(scale)
    return out, out_mag


def rotary(x, weight, positions, inv_freq, start=0, interleaved=False, eps=0.0, scale=1.0):
    x = np.asarray(x, np.float64)
    v, mag = x, np.abs(x)
    if weight is not None:
        rs = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
        v = x * rs * weight
        mag = np.abs(v)
    return _turned(v, mag, positions, inv_freq, start, interleaved, scale, 1.0)


def rotary_backward(x, weight, dout, positions, inv_freq, start=0, interleaved=False, eps=0.0, scale=1.0):
    """(dx, dx_mag, dweight, dweight_mag); the last two None without a weight."""
    d = np.asarray(dout, np.float64)
    u, um = _turned(d, np.abs(d), positions, inv_freq, start, interleaved, scale, -1.0)
    if weight is None:
        return u, um, None, None
    x = np.asarray(x, np.float64)
    rs = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    unit = x * rs
    dw, dw_mag = (u * unit).sum(axis=(0, 1)), (um * np.abs(unit)).sum(axis=(0, 1))
    u, um = u * weight, um * np.abs(weight)
    dx = rs * (u - unit * np.mean(u * unit, axis=-1, keepdims=True))
    dx_mag = rs * (um + np.abs(unit) * np.mean(um * np.abs(unit), axis=-1, keepdims=True))
    return dx, dx_mag, dw, dw_mag


def frequencies(rotary_dim, base, factor=None, original=None, fast=None, slow=None):
    """inv_freq and scale: plain, divided by factor, or by parts."""
    f = [base ** (-2.0 * i / rotary_dim) for i in range(rotary_dim // 2)]
    if original is None:
        return [v / (factor or 1.0) for v in f], 1.0
    turns = [original * v / (2.0 * math.pi) for v in f]      # falls with the index

    def index(n):  # (not whole) index whose frequency makes n turns
        return math.log(turns[0] / n) / math.log(base) * rotary_dim / 2.0

    lo, hi = max(math.floor(index(fast)), 0), min(math.ceil(index(slow)), rotary_dim - 1)
    lo = min(lo, hi - 1)        # all of them are slow, or all fast
    share = [min(max((i - lo) / (hi - lo), 0.0), 1.0) for i in range(rotary_dim // 2)]
    return [v * (1.0 - s) + v / factor * s for v, s in zip(f, share)], 0.1 * math.log(factor) + 1.0
