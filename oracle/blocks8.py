"""64-bit restatements of what a block on 8-bit integers consists of: rows held
in 8 bits, the norms around a block with its gate and residual scale, and the
linear layer, with gradients (definitions in include/sg.h)."""
from __future__ import annotations

import numpy as np

__all__ = ["pack8", "values8", "block_norm_u", "rms", "block_norm_grad", "linear8", "linear8_grad"]

GROUP = 128
MOST = np.float32(float.fromhex("0x1.0204060000000p+121"))  # the largest scale of which 127 are an fp32 number


def pack8(x, group: int):
    """(q, scale) of fp32 values, each step rounded to fp32 as it is defined."""
    x = np.asarray(x, dtype=np.float32)
    rows, cols = x.shape
    w = group or cols
    n = -(-cols // w)
    q = np.zeros((rows, cols), dtype=np.int8)
    scale = np.zeros((rows, n), dtype=np.float32)
    f, least = np.float32, np.float32(2.0 ** -126)
    for r in range(rows):
        for g in range(n):
            v = x[r, g * w:(g + 1) * w]
            if not np.isfinite(v).all():
                scale[r, g] = np.nan
                continue
            a = np.abs(v).max()
            if a < f(127) * least:
                inv, scale[r, g] = f(2.0 ** 126), least if a > 0 else f(0)
            else:
                inv, scale[r, g] = f(1) / a * f(127), min(a * (f(1) / f(127)), MOST)
            q[r, g * w:(g + 1) * w] = np.rint(v * inv)
    return q, scale if group else scale[:, 0]


def values8(q, scale):
    """What 8-bit rows stand for; scale has one for each row or for 128 columns."""
    q, scale = np.asarray(q, dtype=np.float64), np.asarray(scale, dtype=np.float64)
    if scale.ndim == 1:
        return q * scale[:, None]
    return q * np.repeat(scale, GROUP, axis=1)[:, :q.shape[1]]


def rms(x, eps):
    """1 / sqrt(mean of a row's squares + eps)."""
    x = np.asarray(x, dtype=np.float64)
    return 1.0 / np.sqrt((x * x).mean(1) + eps)


def block_norm_u(x, residual, post, gate, alpha, eps):
    """(u before it is rounded, rstd_x)."""
    x, post = np.asarray(x, dtype=np.float64), np.asarray(post, dtype=np.float64)
    r = rms(x, eps)
    u = x * r[:, None] * post
    if gate is not None:
        u = u * np.asarray(gate, dtype=np.float64)
    if residual is not None:
        u = u + alpha * np.asarray(residual, dtype=np.float64)
    return u, r


def block_norm_grad(dy, u, x, post, gate, pre, alpha, rstd_x, rstd_u, du_in=None):
    """dresidual, dx, dpost, dgate, dpre, and du."""
    dy, u, x, post, pre = (np.asarray(a, dtype=np.float64) for a in (dy, u, x, post, pre))
    gate = np.ones_like(post) if gate is None else np.asarray(gate, dtype=np.float64)
    rx, ru = (np.asarray(a, dtype=np.float64)[:, None] for a in (rstd_x, rstd_u))
    m, g = u * ru, dy * pre
    du = ru * (g - m * (g * m).mean(1, keepdims=True))
    if du_in is not None:
        du = du + np.asarray(du_in, dtype=np.float64)
    h, k = x * rx, du * gate * post
    s = (du * h).sum(0)
    return {"dresidual": alpha * du, "dx": rx * (k - h * (k * h).mean(1, keepdims=True)), "dpost": gate * s,
            "dgate": post * s, "dpre": (dy * m).sum(0), "du": du}


def linear8(x8, x_scale, W8, W_scale):
    z = np.asarray(x8, dtype=np.float64) @ np.asarray(W8, dtype=np.float64).T
    return z * np.asarray(x_scale, dtype=np.float64)[:, None] * np.asarray(W_scale, dtype=np.float64)


def linear8_grad(x8, x_scale, W8, W_scale, dout):
    """(dx, dW)"""
    d = np.asarray(dout, dtype=np.float64)
    return d @ values8(W8, W_scale), d.T @ values8(x8, x_scale)
