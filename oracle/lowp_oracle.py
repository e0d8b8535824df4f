"""fp64 definitions of the norm and of the 8-bit operators, in NumPy.

Written from the formulas alone (include/moe.h, "norm and 8-bit operators"); shares no code
with the CUDA library.  Activation scales are [blocks, rows], weight scales
[groups, blocks of N, blocks of K]; e4m3 values are handled as the numbers they stand for.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = E4M3_MAX * 2.0 ** -126


def blocks(n: int) -> int:
    return -(-n // BLOCK)


def e4m3(v):
    """Nearest e4m3 value (ties to even, saturated, NaN kept): 4 significant bits from 2^-6
    on, a fixed step of 2^-9 below."""
    v = np.asarray(v, np.float64)
    _, ex = np.frexp(np.where(np.isfinite(v) & (v != 0), v, 1.0))
    step = np.ldexp(1.0, np.maximum(ex - 1, -6) - 3)
    with np.errstate(invalid="ignore"):
        return np.clip(np.rint(v / step) * step, -E4M3_MAX, E4M3_MAX)


def _blocked(x, axis_blocks):
    pad = axis_blocks * BLOCK - x.shape[-1]
    return np.pad(x, [(0, 0)] * (x.ndim - 1) + [(0, pad)]).reshape(x.shape[:-1] + (axis_blocks, BLOCK))


def quantize_rows(x):
    """(q [rows, d], scale [blocks, rows]); a NaN or an infinity makes its whole block NaN or
    the scale infinite, so that it reads back as NaN."""
    x = np.asarray(x, np.float64)
    v = _blocked(x, blocks(x.shape[1]))
    amax = np.maximum(np.abs(v).max(-1), AMAX_FLOOR)
    with np.errstate(invalid="ignore"):
        q = e4m3(E4M3_MAX * v / amax[..., None])
    return q.reshape(x.shape[0], -1)[:, : x.shape[1]], (amax / E4M3_MAX).T.copy()


def quantize_weights(w):
    """(q, scale) of [groups, N, K]."""
    w = np.asarray(w, np.float64)
    G, N, K = w.shape
    nb, kb = blocks(N), blocks(K)
    p = np.zeros((G, nb * BLOCK, kb * BLOCK))
    p[:, :N, :K] = w
    p = p.reshape(G, nb, BLOCK, kb, BLOCK)
    amax = np.maximum(np.abs(p).max((2, 4)), AMAX_FLOOR)
    with np.errstate(invalid="ignore"):
        q = e4m3(E4M3_MAX * p / amax[:, :, None, :, None])
    return q.reshape(G, nb * BLOCK, kb * BLOCK)[:, :N, :K], amax / E4M3_MAX


def rows_value(q, scale):
    with np.errstate(invalid="ignore"):  # 0 * inf: a block that held an infinity
        return np.asarray(q, np.float64) * np.repeat(np.asarray(scale, np.float64).T, BLOCK, 1)[:, : q.shape[1]]


def weights_value(q, scale):
    s = np.repeat(np.repeat(np.asarray(scale, np.float64), BLOCK, -2), BLOCK, -1)
    return np.asarray(q, np.float64) * s[..., : q.shape[-2], : q.shape[-1]]


def grouped_matmul(a, offsets, b):
    """(out, sum of magnitudes) of rows a [rows, K] times b [groups, N, K]^T by group; rows of
    no group are NaN."""
    out = np.full((a.shape[0], b.shape[1]), np.nan)
    mag = np.full_like(out, np.nan)
    for g in range(b.shape[0]):
        i, j = int(offsets[g]), int(offsets[g + 1])
        out[i:j] = a[i:j] @ b[g].T
        mag[i:j] = np.abs(a[i:j]) @ np.abs(b[g]).T
    return out, mag


def rmsnorm(r, weight, eps):
    """(y, rstd) of the rows r (the sum with the residual already taken)."""
    rstd = 1.0 / np.sqrt(np.mean(r * r, axis=1) + eps)
    return r * rstd[:, None] * weight, rstd


def rmsnorm_backward(r, weight, rstd, dy, dresidual=None):
    """(dx, dweight)."""
    xhat = r * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - xhat * np.mean(g * xhat, axis=1, keepdims=True))
    return dx if dresidual is None else dx + dresidual, (dy * xhat).sum(0)
