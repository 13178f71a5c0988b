"""64-bit restatements of the row-wise operators next to the output layer:
dropout from a counter-based generator and the residual's addition with RMS
norm (definitions in include/sg.h)."""
from __future__ import annotations

import numpy as np

__all__ = ["philox4x32", "dropout_keep", "dropout_scale", "dropout", "add_rmsnorm", "add_rmsnorm_grad"]


def philox4x32(counter, key, rounds: int = 10):
    """Philox4x32 of Salmon et al. (2011) on Python integers: four counter
    words and two key words to four random words."""
    x, k = list(counter), list(key)
    for _ in range(rounds):
        p, q = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [(q >> 32) ^ x[1] ^ k[0], q & 0xFFFFFFFF, (p >> 32) ^ x[3] ^ k[1], p & 0xFFFFFFFF]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return x


def _threshold(p: float) -> int:
    return int(np.floor(p * 65536.0 + 0.5))


def dropout_keep(rows: int, cols: int, p: float, seed: int, offset: int) -> np.ndarray:
    """Which elements of a rows x cols matrix stay."""
    blocks = -(-cols // 8)
    u, m32 = np.uint64, np.uint64(0xFFFFFFFF)
    x = [np.broadcast_to(np.arange(blocks, dtype=u), (rows, blocks)),
         np.broadcast_to(np.arange(rows, dtype=u)[:, None], (rows, blocks)),
         np.full((rows, blocks), offset & 0xFFFFFFFF, dtype=u), np.full((rows, blocks), offset >> 32, dtype=u)]
    k = [seed & 0xFFFFFFFF, seed >> 32]
    for _ in range(10):
        a, b = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(b >> u(32)) ^ x[1] ^ u(k[0]), b & m32, (a >> u(32)) ^ x[3] ^ u(k[1]), a & m32]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    half = np.stack([h for w in x for h in (w & u(0xFFFF), w >> u(16))], axis=-1).reshape(rows, blocks * 8)
    return half[:, :cols] >= u(_threshold(p))


def dropout_scale(p: float) -> np.float32:
    t = _threshold(p)
    return np.float32(65536.0 / (65536 - t)) if t < 65536 else np.float32(0)


def dropout(x: np.ndarray, p: float, seed: int, offset: int) -> np.ndarray:
    """fp32 values after dropout, before any rounding to fewer bits."""
    x = np.asarray(x, dtype=np.float32)
    keep = dropout_keep(x.shape[0], x.shape[1], p, seed, offset)
    return np.where(keep, x * dropout_scale(p), np.float32(0))


def add_rmsnorm(u, weight, eps):
    """(y, rstd) in 64 bits of the rows u as they are stored."""
    u, w = np.asarray(u, dtype=np.float64), np.asarray(weight, dtype=np.float64)
    rstd = 1.0 / np.sqrt((u * u).mean(1) + eps)
    return u * rstd[:, None] * w, rstd


def add_rmsnorm_grad(dy, u, weight, rstd, du_in=None):
    """(du, dweight) in 64 bits, du without dropout."""
    dy, u, w = (np.asarray(a, dtype=np.float64) for a in (dy, u, weight))
    r = np.asarray(rstd, dtype=np.float64)[:, None]
    g, n = dy * w, u * r
    du = r * (g - n * (g * n).mean(1, keepdims=True))
    if du_in is not None:
        du = du + np.asarray(du_in, dtype=np.float64)
    return du, (dy * n).sum(0)
