"""The norms around a block and their gradients in 64 bits (torch, on the
arguments' device), from their formulas, with bounds on what the stated
arithmetic may add: row sums in 64 bits, values in fp32, results rounded once."""
import torch

from int8_reference import EPS, ROUND, TINY, f64

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def rho(v, eps):
    return 1 / torch.sqrt(v.square().mean(1, keepdim=True) + eps)


def state(x, branch, post, gate, alpha, beta, eps, kind):
    """(state, bound). Its terms carry the roundings of rho, of up to four
    products and of the sum."""
    x, v = f64(x), f64(branch)
    if post is not None:
        v = v * rho(v, eps) * f64(post)
    v = beta * v * (1 if gate is None else f64(gate))
    s = alpha * x + v
    return s, ROUND[kind] * s.abs() + 8 * EPS * ((alpha * x).abs() + v.abs()) + TINY[kind]


def normed(s, pre, eps, kind):
    """(y, bound) of a given state: rho, two products."""
    s = f64(s)
    y = s * rho(s, eps) * f64(pre)
    return y, (ROUND[kind] + 4 * EPS) * y.abs() + TINY[kind]


def gradients(s, dout, dy, branch, post, gate, pre, alpha, beta, eps, kind):
    """{name: (gradient, bound)}; gate [N], [M, 1] or [M, N] or None.

    Row sums' terms are fp32 products of two or three factors (3 EPS of each
    term's size), the rest of a sum is exact to 64 bits; sums over tokens are
    fp32 in some order."""
    s = f64(s)
    m, n = s.shape
    zero = torch.zeros_like(s)
    D, E = (zero if dout is None else f64(dout)).clone(), zero.clone()
    E += 2 * EPS * D.abs()
    size = D.abs()
    r = {}
    if dy is not None:
        r1, dy, pre = rho(s, eps), f64(dy), f64(pre)
        unit = s * r1
        terms = (unit * pre * dy)
        c1, c1_abs = terms.mean(1, keepdim=True), terms.abs().mean(1, keepdim=True)
        D = D + r1 * (pre * dy - unit * c1)
        more = r1 * ((pre * dy).abs() + unit.abs() * c1_abs)
        E = E + 8 * EPS * more
        size = size + more
        t = dy * unit
        r["dpre"] = (t.sum(0), (m + 8) * EPS * t.abs().sum(0))
    r["dx"] = (alpha * D, abs(alpha) * E + (ROUND[kind] + EPS) * (alpha * D).abs() + TINY[kind])
    if branch is None:
        return r
    b = f64(branch)
    g = torch.ones(1, 1, dtype=torch.float64, device=s.device) if gate is None else f64(gate)
    if g.dim() == 1:
        g = g[None]
    r2 = rho(b, eps) if post is not None else torch.ones_like(b[:, :1])
    w = f64(post)[None] if post is not None else torch.ones(1, n, dtype=torch.float64, device=s.device)
    unit = b * r2
    v = unit * w
    dv = beta * g * D
    Edv = (beta * g).abs() * E + 4 * EPS * dv.abs()
    db, Edb = dv, Edv
    if post is not None:
        c2 = (v * dv).mean(1, keepdim=True)
        Ec2 = 10 * EPS * (v * beta * g * size).abs().mean(1, keepdim=True)
        db = r2 * (w * dv - unit * c2)
        Edb = r2 * (w.abs() * Edv + unit.abs() * Ec2 + 8 * EPS * ((w * dv).abs() + (unit * c2).abs()))
        t = dv * unit
        r["dpost"] = (t.sum(0), (m + 12) * EPS * t.abs().sum(0) + (unit.abs() * Edv).sum(0))
    r["dbranch"] = (db, Edb + ROUND[kind] * db.abs() + TINY[kind])
    if gate is not None:
        t = beta * D * v
        Et = (beta * v).abs() * E + 6 * EPS * t.abs()
        if f64(gate).dim() == 1:
            r["dgate"] = (t.sum(0), (m + 12) * EPS * t.abs().sum(0) + Et.sum(0))
        elif gate.shape[1] == 1 and (n > 1 or gate.dtype == torch.float32 and kind != "f32"):
            # (the sum of the terms of D, each with the row sums' error)
            r["dgate"] = (t.sum(1, keepdim=True), 10 * EPS * (beta * v * size).abs().sum(1, keepdim=True))
        else:
            r["dgate"] = (t, Et + ROUND[kind] * t.abs() + TINY[kind])
    return r
