"""64-bit restatement of softmax cross entropy of a dense head and its
gradient (definitions in include/sg.h)."""
from __future__ import annotations

import numpy as np

__all__ = ["softmax_ce"]


def softmax_ce(h, W, targets, dloss=None, ignore_index=-100, smoothing=0.0):
    """loss[T] and lse[T]; with dloss[T] also dh and dW and, for error bounds,
    the sums behind each of their elements with g's absolute value in its place
    (_abs) and with the absolute values of g's three parts (_mag)."""
    h, W = np.asarray(h, dtype=np.float64), np.asarray(W, dtype=np.float64)
    y = np.asarray(targets, dtype=np.int64)
    V = W.shape[0]
    live = (y != ignore_index) & (y >= 0) & (y < V)
    z = h @ W.T
    top = z.max(1)
    lse = top + np.log(np.exp(z - top[:, None]).sum(1))
    at = np.where(live, y, 0)
    loss = lse - (1 - smoothing) * z[np.arange(len(y)), at] - smoothing * z.mean(1)
    out = {"loss": np.where(live, loss, 0.0), "lse": lse}
    if dloss is not None:
        c = np.where(live, np.asarray(dloss, dtype=np.float64), 0.0)[:, None]
        g = np.exp(z - lse[:, None])
        mag = g + smoothing / V
        g -= smoothing / V
        g[np.arange(len(y)), at] -= 1 - smoothing
        mag[np.arange(len(y)), at] += 1 - smoothing
        g *= c
        mag *= np.abs(c)
        out["dh"], out["dW"] = g @ W, g.T @ h
        np.abs(g, out=g)
        h, W = np.abs(h), np.abs(W)
        out["dh_abs"], out["dW_abs"] = g @ W, g.T @ h
        out["dh_mag"], out["dW_mag"] = mag @ W, mag.T @ h
    return out
