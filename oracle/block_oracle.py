"""Float64 oracle of what surrounds the products of a decoder block (include/paro_block.h): activations of an
epilogue, the norms around a block, the router and the experts. Test infrastructure only; shares no code with the
library. Values that the definitions hold in a 16-bit or 32-bit type arrive here as exact float64 values.
"""
from __future__ import annotations

import math

import numpy as np

_erfc = np.frompyfunc(math.erfc, 1, 1)


def act(v, kind: str) -> np.ndarray:
    v = np.asarray(v, np.float64)
    with np.errstate(over="ignore", invalid="ignore"):
        if kind == "relu":
            return np.where(v < 0, 0.0, v)
        if kind == "relu2":
            return np.where(v < 0, 0.0, v) ** 2
        if kind == "silu":
            return v / (1.0 + np.exp(-v))
        if kind == "gelu":
            return v * _erfc(-v / math.sqrt(2.0)).astype(np.float64) / 2.0
        if kind == "gelu_tanh":  # (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
            return v / (1.0 + np.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    assert kind == "none"
    return v


def stream(x, residual, eps, post_gamma=None, gate=None, residual_scale=1.0):
    """(h before its rounding to the rows' type, the gated part p of it); gate [B][D], one for M / B rows each."""
    p = np.asarray(x, np.float64)
    if post_gamma is not None:
        p = p * post_gamma / np.sqrt((p * p).mean(axis=1, keepdims=True) + eps)
    if gate is not None:
        p = p * np.repeat(np.atleast_2d(gate), len(p) // len(np.atleast_2d(gate)), axis=0)
    return residual_scale * np.asarray(residual, np.float64) + p, p


def route(x, router, top_k, sigmoid=False, renormalize=True):
    """(ids, weights) of rows x: the largest logits first, the lower index first among equals, NaN last."""
    logits = np.asarray(x, np.float64) @ np.asarray(router, np.float64).T
    with np.errstate(over="ignore", invalid="ignore"):
        key = np.where(np.isnan(logits), -np.inf, logits)
        ids = np.argsort(-key, axis=1, kind="stable")[:, :top_k]
        e = np.exp(logits - key.max(axis=1, keepdims=True))
        score = 1.0 / (1.0 + np.exp(-logits)) if sigmoid else e / e.sum(axis=1, keepdims=True)
        w = np.take_along_axis(score, ids, 1)
        return ids, w / w.sum(axis=1, keepdims=True) if renormalize else w


def silu_mul(g, u):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def experts(x, ids, weights, gate_up, down, between=None):
    """(y, bound of the library's error in y before its last rounding): x [M][D] as the experts see it, gate_up [E][2F][D],
    down [E][D][F] dequantized; between(a): what a goes through before down.

    The bound, with U = 2^-24 and a float32 sum of n exact products off by at most n + 4 roundings of the sum of their
    magnitudes (up to 128 in a group, then one per group, the group's scale and the waves' sums): g and u are off by
    (140 + D / 128) U of theirs; silu has a slope of at most 1.1 and itself costs 4 + |g| roundings; a is rounded to
    float16 (half a step of 2^-11, or 2^-25 below 2^-14); and the down product adds (140 + F / 128) U of its own
    magnitudes, the sum over experts one rounding for each wave and expert (16 + top_k).
    """
    U = 2.0 ** -24
    M, D = x.shape
    F = down.shape[2]
    y, bound = np.zeros((M, D)), np.zeros((M, D))
    for e in range(len(down)):
        takes = ids == e
        at = np.nonzero(takes.any(axis=1))[0]
        if not len(at):
            continue
        w = np.where(takes[at], weights[at], 0.0).sum(axis=1)[:, None]
        gu, mag = x[at] @ gate_up[e].T, np.abs(x[at]) @ np.abs(gate_up[e]).T
        g, u = gu[:, :F], gu[:, F:]
        off = (140 + D // 128) * U * mag
        a = silu_mul(g, u)
        da = 1.1 * np.abs(u) * off[:, :F] + np.abs(g) * off[:, F:] + 1.1 * off[:, :F] * off[:, F:] + (4 + np.abs(g)) * U * np.abs(a)
        da = da + np.maximum(2.0 ** -11 * (np.abs(a) + da), 2.0 ** -25)
        if between is not None:
            a = between(a)
        r = np.abs(down[e]).T
        y[at] += w * (a @ down[e].T)
        bound[at] += np.abs(w) * (da @ r + (160 + len(ids[0]) + F // 128) * U * ((np.abs(a) + da) @ r))
    return y, bound
