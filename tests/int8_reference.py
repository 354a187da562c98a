"""The int8 products and their gradients written out in 64 bits (numpy), from
their formulas, with bounds on what fp32 and 16-bit arithmetic may add."""
import math

import numpy as np

EPS = 2.0 ** -24                       # unit roundoff of fp32
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "f32": 2.0 ** -149}  # half the smallest step

_erf = np.vectorize(math.erf, otypes=[np.float64])


def quantize(x):
    """Codes and scales of the rows of x (any float array), by the stated fp32
    arithmetic."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        top = np.max(np.abs(x), axis=1, initial=0.0)
        scale = np.maximum(top * np.float32(1 / 127), np.float32(2.0 ** -100)).astype(np.float32)
        inv = (np.float32(1) / scale).astype(np.float32)
        q = np.clip(np.rint((x * inv[:, None]).astype(np.float32)), -127, 127)
    bad = ~np.isfinite(x).all(axis=1)
    scale[bad] = np.nan
    q[bad] = 0
    return q.astype(np.int8), scale


def act(name, v):
    """act(v), act'(v)"""
    with np.errstate(over="ignore"):
        if name == "silu":
            p = 1 / (1 + np.exp(-v))
            return v * p, p * (1 + v * (1 - p))
        if name == "gelu":
            p = 0.5 * (1 + _erf(v / math.sqrt(2)))
            return v * p, p + v * np.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        if name == "gelu_tanh":
            c = math.sqrt(2 / math.pi)
            t = np.tanh(c * (v + 0.044715 * v ** 3))
            return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)
    return np.where(v > 0, v, 0.0), (v > 0) * 1.0


def sums(q, w):
    return q.astype(np.int64) @ w.astype(np.int64).T


def gated(q, sx, wg, sg, wu, su, name):
    """H and the fp32 error it may carry: g and u have three roundings each,
    exp an error of its argument's rounding, the rest a few more; 16 EPS
    |g| |u| (1 + |g|) covers them for every activation."""
    sx, sg, su = (np.asarray(v, np.float64) for v in (sx, sg, su))
    g = sums(q, wg) * sx[:, None] * sg
    u = sums(q, wu) * sx[:, None] * su
    return act(name, g)[0] * u, 16 * EPS * np.abs(g) * np.abs(u) * (1 + np.abs(g))


def _dx(d, derr, scales, weights, kind):
    """sum over t of (d_t s_t) w_t with its bound: each d s rounded to 16 bits
    (F16: also to steps of 2^-24 max|s|, below its smallest normal value), fp32
    sums in any order."""
    n = weights[0].shape[0]
    top = max((np.max(np.abs(s), initial=0.0) for s in scales))
    dx, bound = 0.0, 0.0
    for v, e, s, w in zip(d, derr, scales, weights):
        w = w.astype(np.float64)
        dx = dx + (v * s) @ w
        size = np.abs(v * s)
        per = size * (ROUND[kind] + (2 * n + 20) * EPS) + e * np.abs(s)
        if kind == "f16":
            per = per + TINY["f16"] * top
        bound = bound + per @ np.abs(w)
    return dx, bound + ROUND[kind] * np.abs(dx) + TINY[kind]


def gemm_backward(dy, q, sx, w, sw, kind):
    """((dX, bound), (dsw, bound)); dy float64."""
    sx, sw = np.asarray(sx, np.float64), np.asarray(sw, np.float64)
    raw = sums(q, w) * sx[:, None]
    t = dy * raw
    m = len(sx)
    return (_dx([dy], [0 * dy], [sw], [w], kind),
            (t.sum(0), (m + 8) * EPS * np.abs(t).sum(0)))


def gated_backward(dh, q, sx, wg, sg, wu, su, name, kind):
    """((dX, bound), (dsg, bound), (dsu, bound)). act' carries at most
    32 EPS (1 + |g|)^2, act 16 EPS |g| (1 + |g|)."""
    sx, sg, su = (np.asarray(v, np.float64) for v in (sx, sg, su))
    g0, u0 = sums(q, wg) * sx[:, None], sums(q, wu) * sx[:, None]
    g, u = g0 * sg, u0 * su
    a, da = act(name, g)
    dg, du = dh * u * da, dh * a
    eg = np.abs(dh * u) * 32 * EPS * (1 + np.abs(g)) ** 2
    eu = np.abs(dh) * 16 * EPS * np.abs(g) * (1 + np.abs(g))
    m = len(sx)
    ends = [_dx([dg, du], [eg, eu], [sg, su], [wg, wu], kind)]
    for d, e, raw in ((dg, eg, g0), (du, eu, u0)):
        t = d * raw
        ends.append((t.sum(0), (m + 8) * EPS * np.abs(t).sum(0) + (e * np.abs(raw)).sum(0)))
    return ends
