"""The distillation loss from a teacher's top logits and its gradient in 64
bits (torch), from the formulas, with bounds on what the stated arithmetic may
add: exponentials and sums over classes in fp32, the entries' terms in 64
bits, results rounded once."""
import math

import torch

from int8_reference import EPS, ROUND, TINY, f64


def distill(logits, index, teacher, lse=None, weight=None, temperature=1.0, dloss=None, kind="f32"):
    """((loss, bound), (dlogits, bound)); every index below the number of
    classes. The temperature is the fp32 number nearest to the one given."""
    T = float(torch.tensor(temperature, dtype=torch.float32))
    z, t = f64(logits) / T, f64(teacher) / T
    m, v = z.shape
    index = torch.as_tensor(index).long()
    inside = index >= 0
    at = index.clamp_min(0)
    w = torch.ones(m, dtype=torch.float64, device=z.device) if weight is None else f64(weight)
    z = torch.where((w == 0)[:, None], 0, z)  # whatever such a row holds
    t = torch.where(inside, t, -math.inf)
    logp = torch.log_softmax(t, 1) if lse is None else t - f64(lse)[:, None]
    p = torch.where(inside, torch.exp(logp), 0)
    hit = torch.zeros_like(z).scatter_add_(1, at, inside.double()) > 0
    mass = torch.zeros_like(z).scatter_add_(1, at, p)
    L = torch.logsumexp(z, 1, keepdim=True)
    # relative error of an exponential: its argument's three roundings, a few
    # of its own; a sum has a thread's share of the classes and 16 more
    out = z if lse is None else z.masked_fill(hit, -math.inf)
    Lt = torch.logsumexp(out, 1, keepdim=True)
    top = out.amax(1, keepdim=True)
    r = EPS * (4 * (z - torch.where(top.isinf(), 0, top)).abs() + 6)
    share = torch.where(torch.isfinite(out) & torch.isfinite(Lt), torch.exp(out - Lt), 0)
    eL = (share * torch.where(share > 0, r, 0)).sum(1, keepdim=True) + (v / 512 + 24) * EPS
    terms = torch.where(p > 0, p * (torch.where(p > 0, logp, 0) - z.gather(1, at) + L), 0)
    loss, q = terms.sum(1), torch.exp(z - L)
    # (L has the coefficient sum p, and pt with a tail: not 1 where sum p is above
    # 1, or below it with entries that cover every class)
    total = p.sum(1, keepdim=True)
    any_ = inside.any(1)
    if lse is not None:
        pt = (1 - p.sum(1)).clamp_min(0)
        pt = torch.where(hit.all(1), 0, pt)[:, None]
        total = total + pt
    g = total * q - mass
    size = total * q + mass
    if lse is not None:
        loss = loss + torch.where(pt > 0, pt * (pt.clamp_min(1e-300).log() - Lt + L), 0)[:, 0]
        g = torch.where(hit, g, total * q - pt * share)
        size = size + pt * share
    g, size = (torch.where(any_[:, None], x, 0) for x in (g, size))
    loss = torch.where(any_ & (w != 0), loss * w, 0)
    by = w / T * (1 if dloss is None else f64(dloss))
    g = g * by[:, None]
    # (the terms' own rounding in 64 bits: 1e-13 of their size)
    big = torch.where(p > 0, p * (torch.where(p > 0, logp, 0).abs() + z.gather(1, at).abs() + L.abs()), 0).sum(1)
    lb = w.abs() * (2 * eL[:, 0] + 1e-13 * big) + 2 * EPS * loss.abs() + 2.0 ** -149
    gb = by.abs()[:, None] * size * (torch.where(size > 0, r, 0) + 3 * eL + 16 * EPS) + ROUND[kind] * g.abs() + TINY[kind]
    return (loss, lb), (g, gb)
