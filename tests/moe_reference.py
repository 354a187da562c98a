"""The mixture-of-experts layer in 64 bits (torch), from its formulas, with a
bound on what fp32 arithmetic may add: hidden values carry the error of the
gated product, and one whose place between two codes is nearer to a border
than that may get the neighbouring code."""
import numpy as np
import torch

from int8_reference import EPS, ROUND, TINY, f64, gated, quantize, sums


def choose(x, router, top_k, normalize):
    """(experts [M, k], p [M, k]): ties go to the lowest index, NaN first."""
    l = (f64(x)[:, None, :] * f64(router)[None]).sum(2)
    order = torch.where(l.isnan(), torch.inf, l)
    at = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :top_k]
    p = torch.softmax(l, 1).gather(1, at)
    if normalize:
        p = torch.softmax(l.gather(1, at), 1)
    return at, p


def layer(x, router, gate, sg, up, su, down, sd, top_k, act, normalize, kind):
    """(experts, p, y, bound); everything on the CPU or on one device."""
    at, p = choose(x, router, top_k, normalize)
    m, e, n = x.shape[0], gate.shape[0], down.shape[1]
    q, sx = quantize(x.float().cpu().numpy())
    q, sx = torch.from_numpy(q).to(x.device), torch.from_numpy(sx).to(x.device)
    y = torch.zeros(m, n, dtype=torch.float64, device=x.device)
    bound, used = torch.zeros_like(y), len(torch.unique(at))
    for i in range(e):
        who, place = (at == i).nonzero(as_tuple=True)
        if not len(who):
            continue
        h, eh = gated(q[who], sx[who], gate[i], sg[i], up[i], su[i], act)
        top = h.abs().amax(1, keepdim=True)
        sh = torch.clamp(top * float(np.float32(1 / 127)), min=2.0 ** -100)
        rel = eh.amax(1, keepdim=True) / top.clamp_min(1e-300) + 4 * EPS  # of the scale
        v = h / sh
        code = v.round().clamp(-127, 127)
        off = eh / sh + v.abs() * rel + 1e-300
        border = (v - v.floor() - 0.5).abs()  # how far the value is from the nearest half
        flips = (border <= off).double()
        w = f64(down[i])
        f = (p[who, place][:, None] * sh) * f64(sd[i]).abs()[None]
        y[who] += p[who, place][:, None] * sh * f64(sd[i])[None] * (code @ w.T)
        size = code.abs() @ w.abs().T
        bound[who] += f * (flips @ w.abs().T + size * (rel + (used + 20) * EPS))
    return at, p, y, bound + ROUND[kind] * y.abs() + TINY[kind]
