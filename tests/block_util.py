"""Runs the operators around the layer on torch tensors for the tests.

Tolerances: an output of the reference comes with the magnitude of its terms
(oracle/block.py).  A float32 implementation of the same formula rounds each
of them a few times and adds them in some order; ``near`` takes the number of
such roundings, u = 2^-24 each, and half a step of the output's own type
(2^-8 for BF16, 2^-24 for float32).
"""

from __future__ import annotations

import numpy as np
import torch

from fp8_mixture_experts_amd import binding as B

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
TYPE = {torch.bfloat16: B.MEGA_MOE_BF16, torch.float32: B.MEGA_MOE_F32}
KIND = {"none": B.MEGA_MOE_GATE_NONE, "token": B.MEGA_MOE_GATE_TOKEN, "channel": B.MEGA_MOE_GATE_CHANNEL,
        "full": B.MEGA_MOE_GATE_FULL}
SCORE = {"softmax": B.MEGA_MOE_SCORE_SOFTMAX, "sigmoid": B.MEGA_MOE_SCORE_SIGMOID}


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def near(got, want, mag, roundings, label=""):
    """got (a tensor) within half a step of its type and `roundings` of float32."""
    half = HALF[got.dtype]
    g = f64(got)
    assert g.shape == np.shape(want), (label, g.shape, np.shape(want))
    err = roundings * U * np.asarray(mag)
    limit = (1 + half) * err + half * np.abs(want) + 2.0 ** -133
    off = np.abs(g - want)
    bad = ~(off <= limit)
    assert not bad.any(), (f"{label}: {int(bad.sum())} of {bad.size} outside, worst "
                           f"{float((off / limit)[bad].max()):.3g} of the limit, at {np.argwhere(bad)[:3].tolist()}")


def current_stream():
    return torch.cuda.current_stream().cuda_stream


def padded(rows, cols, dtype, extra, fill=7.0):
    """A [rows, cols] view whose rows lie `extra` elements apart, and its whole
    buffer, filled."""
    buf = torch.full((rows, cols + extra), fill, dtype=dtype, device="cuda")
    return buf[:, :cols], buf


def workspace(nbytes):
    """A workspace of exactly the bytes asked for, full of NaN patterns."""
    assert nbytes >= 0
    t = torch.full((max(nbytes, 16),), 0xFF, dtype=torch.uint8, device="cuda")
    return {"workspace": t, "workspace_bytes": nbytes}


def finish_norm_backward(a, stream=None):
    B.set_args(a, **workspace(B.mega_moe_norm_workspace_bytes(a)))
    B.mega_moe_norm_backward(a, current_stream() if stream is None else stream)


def codes(q):
    """E4M3 bytes as values."""
    return q.view(torch.float8_e4m3fn).float().cpu().double().numpy()
