"""The int8 products and their gradients written out in 64 bits (torch, on
whatever device the arguments are), from their formulas, with bounds on what
fp32 and 16-bit arithmetic may add. Arguments are numpy arrays or tensors."""
import math

import numpy as np
import torch

EPS = 2.0 ** -24                       # unit roundoff of fp32
ROUND = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -133, "f16": 2.0 ** -25, "f32": 2.0 ** -149}  # half the smallest step


def f64(a):
    return torch.as_tensor(a).double()


def quantize(x):
    """Codes and scales of the rows of x (any float array), by the stated fp32
    arithmetic, in numpy."""
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
    v = f64(v)
    if name == "silu":
        p = 1 / (1 + torch.exp(-v))
        return v * p, p * (1 + v * (1 - p))
    if name == "gelu":
        p = 0.5 * torch.erfc(-v / math.sqrt(2))
        return v * p, p + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v ** 3))
        return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 3 * 0.044715 * v * v)
    return torch.where(v > 0, v, 0 * v), (v > 0) * 1.0


def sums(q, w):
    return f64(q) @ f64(w).T  # exact: every sum is an integer below 2^31


def gated(q, sx, wg, sg, wu, su, name):
    """H and the fp32 error it may carry: g and u have three roundings each,
    exp an error of its argument's rounding, the rest a few more; 16 EPS
    |g| |u| (1 + |g|) covers them for every activation."""
    sx, sg, su = f64(sx), f64(sg), f64(su)
    g = sums(q, wg) * sx[:, None] * sg
    u = sums(q, wu) * sx[:, None] * su
    return act(name, g)[0] * u, 16 * EPS * g.abs() * u.abs() * (1 + g.abs())


def _dx(d, derr, scales, weights, kind):
    """sum over t of (d_t s_t) w_t with its bound: each d s rounded to 16 bits
    (F16: also to steps of 2^-24 max|s|, below its smallest normal value), fp32
    sums in any order."""
    n = weights[0].shape[0]
    top = max(float(s.abs().max()) for s in scales) if n else 0.0
    dx, bound = 0.0, 0.0
    for v, e, s, w in zip(d, derr, scales, weights):
        w = f64(w)
        dx = dx + (v * s) @ w
        per = (v * s).abs() * (ROUND[kind] + (2 * n + 20) * EPS) + e * s.abs()
        if kind == "f16":
            per = per + TINY["f16"] * top
        bound = bound + per @ w.abs()
    return dx, bound + ROUND[kind] * dx.abs() + TINY[kind]


def gemm_backward(dy, q, sx, w, sw, kind):
    """((dX, bound), (dsw, bound)); dy float64."""
    dy, sx, sw = f64(dy), f64(sx), f64(sw)
    t = dy * (sums(q, w) * sx[:, None])
    m = len(sx)
    return (_dx([dy], [0 * dy], [sw], [w], kind),
            (t.sum(0), (m + 8) * EPS * t.abs().sum(0)))


def gated_backward(dh, q, sx, wg, sg, wu, su, name, kind):
    """((dX, bound), (dsg, bound), (dsu, bound)). act' carries at most
    32 EPS (1 + |g|)^2, act 16 EPS |g| (1 + |g|)."""
    dh, sx, sg, su = f64(dh), f64(sx), f64(sg), f64(su)
    g0, u0 = sums(q, wg) * sx[:, None], sums(q, wu) * sx[:, None]
    g, u = g0 * sg, u0 * su
    a, da = act(name, g)
    dg, du = dh * u * da, dh * a
    eg = (dh * u).abs() * 32 * EPS * (1 + g.abs()) ** 2
    eu = dh.abs() * 16 * EPS * g.abs() * (1 + g.abs())
    m = len(sx)
    ends = [_dx([dg, du], [eg, eu], [sg, su], [wg, wu], kind)]
    for d, e, raw in ((dg, eg, g0), (du, eu, u0)):
        t = d * raw
        ends.append((t.sum(0), (m + 8) * EPS * t.abs().sum(0) + (e * raw.abs()).sum(0)))
    return ends
