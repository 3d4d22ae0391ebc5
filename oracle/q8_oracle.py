"""Float64 oracle of the 8-bit path (include/paro_w8a8.h): row quantiser, residual RMS norm, weight
fold and the W8A8 products. Test infrastructure only; shares no code with the library. Values that
the definitions hold in a 16-bit or 32-bit type arrive here as exact float64 values.
"""
from __future__ import annotations

import numpy as np

from .paro_oracle import transform_activations

TOP_MIN = 2.0 ** -100


def round_to(a, dtype: str) -> np.ndarray:
    """float64 -> the nearest value of 'f16', 'bf16' or 'f32' (ties to even), as float64."""
    a = np.asarray(a, np.float64)
    if dtype == "f32":
        return a.astype(np.float32).astype(np.float64)
    bits, emin, top = (11, -14, 65504.0) if dtype == "f16" else (8, -126, 2.0 ** 127 * (2 - 2.0 ** -7))
    with np.errstate(invalid="ignore", divide="ignore"):
        e = np.maximum(np.frexp(a)[1] - 1, emin)
        step = np.ldexp(1.0, e - (bits - 1))
        r = np.where(np.isfinite(a), np.rint(a / step) * step, a)
    return np.where(np.abs(r) > top, np.copysign(np.inf, r), r)


def quantize_exact(v):
    """(real-valued codes v * 127 / c, scales) of rows v, before any rounding: c = max(max|v|, 2^-100)."""
    v = np.asarray(v, np.float64)
    c = np.maximum(np.abs(v).max(axis=1), TOP_MIN)
    return v * 127.0 / c[:, None], c / 127.0


def rmsnorm(h, gamma, eps):
    """n = h gamma / sqrt(mean(h^2) + eps), in float64."""
    h = np.asarray(h, np.float64)
    return h * np.asarray(gamma, np.float64) / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)


def transform(x, pairs, theta, scale):
    """The activation-side transform in float64 (no rounding to 16 bits)."""
    return transform_activations(np.asarray(x, np.float64), pairs, theta, scale)


def pack_weights(W, pairs=None, theta=None, scale=None):
    """Codes and scales of the (folded) weight rows: the stages in order, then times s, every operation
    rounded on its own in float64; code = rint(b * 127 / c) of the exact quotient (in 64 digits, where a
    value half way between two codes stays there) and scale = float32(c / 127)."""
    b = np.array(W, np.float64)
    if pairs is not None:
        for pk, tk in zip(pairs, theta):
            c = np.cos(np.asarray(tk, np.float64)).astype(np.float32).astype(np.float64)
            s = np.sin(np.asarray(tk, np.float64)).astype(np.float32).astype(np.float64)
            i, j = pk[:, 0], pk[:, 1]
            bi, bj = b[:, i].copy(), b[:, j].copy()
            b[:, i] = c * bi + s * bj
            b[:, j] = c * bj - s * bi
        b = b * np.asarray(scale, np.float32).astype(np.float64)
    c = np.maximum(np.abs(b).max(axis=1), TOP_MIN)
    assert np.finfo(np.longdouble).nmant >= 63
    q = np.rint(b.astype(np.longdouble) * 127 / c.astype(np.longdouble)[:, None])
    return q.astype(np.int8), (c / 127.0).astype(np.float32)


def linear(xq, xs, wq, ws):
    """xs ws sum xq wq in float64 (the integer sum is exact: below 2^53)."""
    acc = np.asarray(xq, np.float64) @ np.asarray(wq, np.float64).T
    return acc * np.asarray(xs, np.float64)[:, None] * np.asarray(ws, np.float64)


def gated(xq, xs, wq, ws):
    """(silu(g) u, g, u): the first half of the rows of wq is the gate."""
    y = linear(xq, xs, wq, ws)
    g, u = y[:, : y.shape[1] // 2], y[:, y.shape[1] // 2:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u, g, u
