"""The operators around a compressed block measured: the RMS norms before and
after a block with its gate and residual scale (forward and backward), the
distillation loss from a teacher's top logits (the loss alone, and with the
gradient of the logits), and a mixture-of-experts layer on int8 codes for few
tokens.

A case's fields: op ("norm", "distill" or "moe"), back (the backward pass), t
(the activations' or logits' type), m tokens.
norm: n channels; branch (a block's output joins the residual), post (it is
normalised first), gate ("", "channel", "token" or "full": one factor for each
channel, for each token, or for each value), y ("", "t" or "codes": the norm
before the next block, in the activations' type or as int8 codes).
distill: v classes, k entries of the teacher's, tail (the mass outside them is
a class of its own), ragged (tokens with fewer entries, and tokens of weight
0), wide (64-bit indices).
moe: e experts, k of them for a token, d channels, f hidden channels, act,
norm (softmax over the chosen experts, else over all), r (the router's type)."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("silu", "gelu", "gelu_tanh", "relu")
EPS = 1e-6
ALPHA, BETA = 0.875, 1.25
TEMPERATURE = 1.5


def _norm(name, m, n, t, gate, y, back=False, branch=True, post=True):
    return {"name": name, "op": "norm", "back": back, "m": m, "n": n, "t": t, "branch": branch,
            "post": post, "gate": gate, "y": y}


def _distill(name, m, v, k, t, back, tail, ragged, wide):
    return {"name": name, "op": "distill", "back": back, "m": m, "v": v, "k": k, "t": t,
            "tail": tail, "ragged": ragged, "wide": wide}


def _moe(name, m, e, k, d, f, t, r, act, norm):
    return {"name": name, "op": "moe", "back": False, "m": m, "e": e, "k": k, "d": d, "f": f,
            "t": t, "r": r, "act": act, "norm": norm}


def listed():
    return [
        # one generated token between two blocks, codes for the next product: the smallest call
        _norm("norm_token", 1, 8192, "bf16", "", "codes"),
        # a short prompt with odd sides and a factor for every value, codes for the next product
        _norm("norm_ragged", 333, 5121, "f16", "full", "codes"),
        # a long prompt between two blocks, with a factor per channel
        _norm("norm_prompt", 4096, 8192, "bf16", "channel", "t"),
        # a short sequence in training, a factor for each token
        _norm("norm_back_short", 96, 5120, "f16", "token", "t", back=True),
        # a training batch of tokens, all gradients
        _norm("norm_back", 4096, 8192, "bf16", "channel", "t", back=True),
        # the loss of a few tokens of an evaluation, fp32 logits
        _distill("distill_few", 7, 32000, 16, "f32", False, True, False, True),
        # the loss of an evaluation batch
        _distill("distill_loss", 4096, 32000, 64, "bf16", False, False, True, False),
        # a short training batch over an odd vocabulary, the tail's mass kept
        _distill("distill_back_ragged", 515, 50021, 20, "f16", True, True, True, True),
        # a training batch: the loss and its gradient
        _distill("distill_back", 4096, 32000, 64, "bf16", True, True, False, False),
        # one generated token, few large experts
        _moe("moe_token", 1, 8, 2, 5120, 13824, "bf16", "f32", "silu", True),
        # four sequences in step, many small experts
        _moe("moe_small", 4, 64, 6, 2048, 1024, "f16", "f16", "gelu_tanh", False),
        # 48 sequences in step, every expert in use: the largest case
        _moe("moe_batch", 48, 64, 6, 5120, 1728, "bf16", "bf16", "silu", True),
    ]


def draw(rng):
    def spread(lo, hi):
        return round(math.exp(rng.uniform(math.log(lo), math.log(hi))))

    def side(lo, hi):
        step = rng.choice((64, 64, 16, 1))
        return max(step, spread(lo, hi) // step * step)

    while True:
        op = rng.choice(("norm", "norm", "distill", "distill", "moe"))
        t = rng.choice(("bf16", "bf16", "f16", "f32"))
        if op == "norm":
            branch = rng.random() < 0.8
            c = {"op": op, "back": rng.random() < 0.5, "m": spread(1, 4096), "n": side(256, 16384),
                 "t": t, "branch": branch, "post": branch and rng.random() < 0.7,
                 "gate": rng.choice(("", "channel", "token", "full")) if branch else "",
                 "y": rng.choice(("", "t", "codes")) if branch else rng.choice(("t", "codes"))}
            if c["back"] and c["y"] == "codes":
                c["y"] = "t"  # (the gradient is the same)
            limit = 4.1e8
        elif op == "distill":
            c = {"op": op, "back": rng.random() < 0.6, "m": spread(1, 4096), "v": side(1000, 131072),
                 "k": spread(1, 128), "t": t, "tail": rng.random() < 0.5,
                 "ragged": rng.random() < 0.5, "wide": rng.random() < 0.5}
            limit = 5.2e8
        else:
            e = rng.choice((4, 8, 16, 32, 60, 64, 128))
            c = {"op": op, "back": False, "m": rng.choice((1, 1, spread(1, 64))), "e": e,
                 "k": rng.randint(1, min(8, e)), "d": side(512, 8192), "f": side(256, 13824),
                 "t": rng.choice(("bf16", "bf16", "f16")), "r": rng.choice(("f32", "t")),
                 "act": rng.choice(ACTS), "norm": rng.random() < 0.5}
            c["r"] = c["t"] if c["r"] == "t" else "f32"
            # (the codes of all experts lie in memory, whatever a token takes of them)
            limit = 1.75e9 if 3 * e * c["d"] * c["f"] <= 4e9 else 0
        if work(c)["bytes"] <= limit:
            return c


def _active(case):
    """Experts that m tokens of k each are expected to use."""
    e = case["e"]
    return e * (1 - (1 - case["k"] / e) ** case["m"])


def work(case):
    m, b = case["m"], BYTES[case["t"]]
    if case["op"] == "norm":
        n = case["n"]
        gate = {"": 0, "channel": 4 * n, "token": 4 * m, "full": m * n * b}[case["gate"]]
        small = 4 * n * (bool(case["y"]) + case["post"])
        if case["back"]:
            # s, the branch and the incoming gradients in, their gradients out
            values = 1 + bool(case["y"]) + 1 + (3 if case["branch"] else 0)
            return {"bytes": values * m * n * b + 2 * (small + gate), "flops": 24 * m * n}
        y = {"": 0, "t": m * n * b, "codes": m * n + 4 * m}[case["y"]]
        values = 3 if case["branch"] else 1
        return {"bytes": values * m * n * b + y + small + gate, "flops": 10 * m * n}
    if case["op"] == "distill":
        top = m * case["k"] * ((8 if case["wide"] else 4) + 4)
        rows = m * case["v"] * b
        return {"bytes": rows * (2 if case["back"] else 1) + top + 12 * m,
                "flops": m * case["v"] * (6 if case["back"] else 4)}
    d, f = case["d"], case["f"]
    weights = _active(case) * (3 * d * f + 4 * (2 * f + d)) + case["e"] * d * BYTES[case["r"]]
    return {"bytes": weights + 2 * m * d * b + 8 * m * case["k"],
            "flops": 6 * m * case["k"] * d * f + 2 * m * case["e"] * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _states(m, n, g):
    """Hidden states: normal, with channels of very different size and a few
    that stand far out."""
    size = torch.exp(0.5 * torch.randn(n, device="cuda", generator=g))
    size[torch.rand(n, device="cuda", generator=g) < 0.002] *= 10
    return torch.randn(m, n, device="cuda", generator=g) * size


def _codes(e, n, k, g):
    """[e, n, k] codes as a weight quantiser leaves them (Laplacian, a few bits
    of entropy) and a positive scale per row."""
    codes = torch.empty(e * n, k, dtype=torch.int8, device="cuda")
    for r in range(0, e * n, 16384):
        v = torch.empty(min(16384, e * n - r), k, device="cuda").exponential_(1.0, generator=g)
        s = torch.rand(v.shape, device="cuda", generator=g)
        codes[r:r + v.shape[0]] = (torch.where(s < 0.5, -v, v) * 2.0).round().clamp(-127, 127)
    scales = 0.35 / math.sqrt(k) * torch.exp(0.3 * torch.randn(e, n, device="cuda", generator=g))
    return codes.view(e, n, k), scales


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m, t = case["m"], TYPES[case["t"]]
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    new = lambda *shape, dtype=t: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    s = {"case": case}
    if case["op"] == "norm":
        n = case["n"]
        s["x"] = _states(m, n, g).to(t)
        s["branch"] = (0.5 * _states(m, n, g)).to(t) if case["branch"] else None
        s["post"] = 1 + 0.2 * rand(n) if case["post"] else None
        s["gate"] = {"": lambda: None, "channel": lambda: 0.5 + 0.2 * rand(n),
                     "token": lambda: torch.sigmoid(rand(m, 1)),
                     "full": lambda: torch.sigmoid(rand(m, n)).to(t)}[case["gate"]]()
        s["pre"] = 1 + 0.2 * rand(n) if case["y"] else None
        if case["back"]:
            # (fp16 training scales its loss, the others do not)
            size = 1.0 if case["t"] == "f16" else 1e-3
            s["dout"] = (size * rand(m, n)).to(t)
            s["dy"] = (size * rand(m, n)).to(t) if case["y"] else None
            s["dx"] = new(m, n)
            s["dbranch"] = new(m, n) if case["branch"] else None
            s["dgate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
            s["dpre"] = new(n, dtype=torch.float32) if case["y"] else None
            s["dpost"] = new(n, dtype=torch.float32) if case["post"] else None
        else:
            s["out"] = new(m, n) if case["branch"] else None
            s["y"] = {"": lambda: None, "t": lambda: new(m, n),
                      "codes": lambda: new(m, n, dtype=torch.int8)}[case["y"]]()
            s["scales"] = new(m, dtype=torch.float32) if case["y"] == "codes" else None
            # (16 bits: a code next to a border may be one off, as after any rounding before it)
            values = torch.bfloat16 if case["t"] == "f32" else t
            s["values"] = new(m, n, dtype=values) if case["y"] == "codes" else None
    elif case["op"] == "distill":
        v, k = case["v"], case["k"]
        # logits of a trained model: a few classes far above the rest
        full = 2.5 * rand(m, v)
        full[:, :min(32, v)] += 6.0 * torch.rand(m, min(32, v), device="cuda", generator=g)
        s["teacher"], index = torch.topk(full, min(k, v), dim=1)
        s["lse"] = torch.logsumexp(full / TEMPERATURE, 1) if case["tail"] else None
        s["logits"] = full.add_(0.8 * rand(m, v)).to(t)
        s["weight"] = None
        if case["ragged"]:
            s["weight"] = torch.where(torch.rand(m, device="cuda", generator=g) < 0.3, 0.0, 1.0)
            entries = torch.randint(1, k + 1, (m, 1), device="cuda", generator=g)
            index[torch.arange(index.shape[1], device="cuda") >= entries] = -1
        s["index"] = index if case["wide"] else index.to(torch.int32)
        s["loss"] = new(m, dtype=torch.float32)
        if case["back"]:
            s["dloss"] = torch.full((m,), 1.0 if case["t"] == "f16" else 1.0 / m, device="cuda")
            s["dlogits"] = new(m, v)
    else:
        e, d, f = case["e"], case["d"], case["f"]
        s["x"] = _states(m, d, g).to(t)
        # (some spread of the logits, whatever the channels' number)
        s["router"] = (rand(e, d) * (2.0 / math.sqrt(d))).to(TYPES[case["r"]])
        s["w"] = [*_codes(e, f, d, g), *_codes(e, f, d, g), *_codes(e, d, f, g)]
        s["y"] = new(m, d)
        s["experts"] = new(m, case["k"], dtype=torch.int32)
        s["weights"] = new(m, case["k"], dtype=torch.float32)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _rho(v):
    return torch.rsqrt(v.square().mean(1, keepdim=True) + EPS)


def _quantise(x):
    """Codes and scales of the rows of x, in 32 bits."""
    scale = (x.abs().amax(1) * torch.tensor(1 / 127, dtype=torch.float32)).clamp_min(2.0 ** -100)
    inv = torch.reciprocal(scale)
    return (x * inv[:, None]).round().clamp(-127, 127), scale


def _plain_norm(s):
    case, t = s["case"], TYPES[s["case"]["t"]]
    out, y, state = None, None, s["x"].float()
    if case["branch"]:
        v = s["branch"].float()
        if case["post"]:
            v = v * _rho(v) * s["post"]
        if s["gate"] is not None:
            v = v * s["gate"].float()
        out = (ALPHA * state + BETA * v).to(t)
        state = out.float()
    if case["y"] == "t":
        y = (state * _rho(state) * s["pre"]).to(t)
    if case["y"] == "codes":
        q, scale = _quantise(state * s["pre"])
        y = (q * (scale[:, None] * _rho(state))).to(s["values"].dtype)
    return out, y


def _plain_norm_back(s):
    case, t = s["case"], TYPES[s["case"]["t"]]
    state, d, dpre = s["x"].float(), s["dout"].float(), None
    if case["y"]:
        rho, dy = _rho(state), s["dy"].float()
        scaled = dy * s["pre"]
        d = d + rho * (scaled - state * rho.square() * (state * scaled).mean(1, keepdim=True))
        dpre = (dy * state * rho).sum(0)
    if not case["branch"]:
        return d.to(t), None, None, dpre, None
    dx = (ALPHA * d).to(t)
    d = BETA * d
    b = s["branch"].float()
    unit = b * _rho(b) if case["post"] else b
    dgate, dpost = None, None
    if s["gate"] is not None:
        dgate = d * (unit * s["post"] if case["post"] else unit)
        dgate = {"channel": lambda: dgate.sum(0), "token": lambda: dgate.sum(1, keepdim=True),
                 "full": lambda: dgate.to(t)}[case["gate"]]()
        d = d * s["gate"].float()
    if case["post"]:
        dpost = (d * unit).sum(0)
        d = d * s["post"]
        d = _rho(b) * (d - unit * (d * unit).mean(1, keepdim=True))
    return dx, d.to(t), dgate, dpre, dpost


def _plain_distill(s):
    case = s["case"]
    z = s["logits"].float() / TEMPERATURE
    there = s["index"] >= 0
    index = torch.where(there, s["index"], 0).long()
    # the terms of the loss nearly cancel: its few entries are computed in 64 bits
    top = s["teacher"].double() / TEMPERATURE
    if case["tail"]:
        mark = torch.zeros_like(z).scatter_add_(1, index, there.float()) > 0  # the teacher's classes
        logp = torch.where(there, top - s["lse"].double()[:, None], -math.inf)
        rest = z.masked_fill(mark, -math.inf)
    else:
        logp = torch.log_softmax(torch.where(there, top, -math.inf), 1)
        rest = z
    p = torch.exp(logp)
    most = z.amax(1, keepdim=True)
    lse = most.double() + z.sub(most).exp_().sum(1, dtype=torch.float64, keepdim=True).log()
    chosen = s["logits"].gather(1, index).double() / TEMPERATURE
    terms = torch.where(there, p * (torch.where(there, logp, 0) - chosen + lse), 0)
    loss = terms.sum(1)
    if case["tail"]:
        pt = (1 - p.sum(1)).clamp_min(0)
        peak = rest.amax(1, keepdim=True)
        lt = peak.double() + rest.sub(peak).exp_().sum(1, dtype=torch.float64, keepdim=True).log()
        log_qt = (lt - lse).squeeze(1)
        loss = loss + torch.where(pt > 0, pt * (pt.clamp_min(1e-300).log() - log_qt), 0)
    weight = torch.ones_like(loss) if s["weight"] is None else s["weight"].double()
    loss = torch.where(weight == 0, 0, loss * weight).float()
    if not case["back"]:
        return loss
    if case["tail"]:
        d = rest.sub_(lt.float()).exp_().mul_((log_qt.exp() - pt).float()[:, None])
        d = torch.where(mark, (z - lse.float()).exp_(), d)
    else:
        d = z.sub_(lse.float()).exp_()
    d.scatter_add_(1, index, torch.where(there, -p, 0).float())
    d *= (weight * s["dloss"].double() / TEMPERATURE).float()[:, None]
    d = torch.where(weight[:, None] == 0, 0, d)
    return loss, d.to(s["logits"].dtype)


def _act(name, v):
    if name == "silu":
        return v / (1 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return torch.where(v > 0, v, 0)


def _plain_moe(s):
    case, x = s["case"], s["x"]
    m, f, d = case["m"], case["f"], case["d"]
    gate, gate_scales, up, up_scales, down, down_scales = s["w"]
    logits = x.double() @ s["router"].double().t()  # choices are made next to a border
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    experts = order.indices[:, :case["k"]]
    over = order.values[:, :case["k"]] if case["norm"] else logits
    weights = torch.exp(order.values[:, :case["k"]] - torch.logsumexp(over, 1, keepdim=True)).float()
    used = torch.unique(experts)
    share = torch.zeros(m, case["e"], device="cuda").scatter_(1, experts, weights)[:, used]
    q, sx = _quantise(x.float())
    qt = q.t().contiguous()
    g = (gate[used].float().view(-1, d) @ qt).view(-1, f, m) * gate_scales[used][:, :, None] * sx
    u = (up[used].float().view(-1, d) @ qt).view(-1, f, m) * up_scales[used][:, :, None] * sx
    h = _act(case["act"], g) * u
    sh = (h.abs().amax(1, keepdim=True) * torch.tensor(1 / 127, dtype=torch.float32)).clamp_min(2.0 ** -100)
    qh = (h * torch.reciprocal(sh)).round().clamp(-127, 127)
    o = torch.bmm(down[used].float(), qh) * sh * down_scales[used][:, :, None]  # [used, d, m]
    y = (o * share.t()[:, None, :]).sum(0)
    return y.t().contiguous().to(x.dtype), experts.to(torch.int32), weights


def _plain(s):
    case = s["case"]
    if case["op"] == "norm":
        return (_plain_norm_back if case["back"] else _plain_norm)(s)
    return _plain_distill(s) if case["op"] == "distill" else _plain_moe(s)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------

def _own(s):
    case = s["case"]
    if case["op"] == "norm":
        from entropy_coded_weight_amd import norm
        if case["back"]:
            norm.block_backward(s["x"], s["dout"], s["dy"], s["branch"], s["post"], s["gate"],
                                s["pre"], s["dx"], s["dbranch"], s["dgate"], s["dpre"], s["dpost"],
                                alpha=ALPHA if case["branch"] else 1.0,
                                beta=BETA if case["branch"] else 1.0, eps=EPS)
            return s["dx"], s["dbranch"], s["dgate"], s["dpre"], s["dpost"]
        norm.block(s["x"], s["branch"], s["out"], s["post"], s["gate"], s["pre"], s["y"],
                   s["scales"], alpha=ALPHA if case["branch"] else 1.0,
                   beta=BETA if case["branch"] else 1.0, eps=EPS)
        if case["y"] == "codes":
            return s["out"], torch.mul(s["y"], s["scales"][:, None], out=s["values"])
        return s["out"], s["y"]
    if case["op"] == "distill":
        from entropy_coded_weight_amd import distill
        if case["back"]:
            distill.loss_backward(s["logits"], s["index"], s["teacher"], s["dlogits"], s["dloss"],
                                  s["loss"], s["lse"], s["weight"], TEMPERATURE)
            return s["loss"], s["dlogits"]
        distill.loss(s["logits"], s["index"], s["teacher"], s["loss"], s["lse"], s["weight"],
                     TEMPERATURE)
        return s["loss"]
    from entropy_coded_weight_amd import moe
    moe.few(s["x"], s["router"], *s["w"], s["y"], case["k"], case["act"], case["norm"],
            s["experts"], s["weights"])
    return s["y"], s["experts"], s["weights"]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# in 64 bits
# ---------------------------------------------------------------------------

def _rms(v):
    return v / torch.sqrt((v * v).sum(1, keepdim=True) / v.shape[1] + EPS)


def _exact_norm(s, case):
    t = TYPES[case["t"]]
    f = {k: v.double() for k, v in s.items() if k in ("x", "branch", "post", "gate", "pre") and v is not None}
    back = case["back"]
    if back:
        f = {k: v.requires_grad_() for k, v in f.items()}

    def added():  # what the branch adds to the residual
        v = f["branch"]
        if "post" in f:
            v = _rms(v) * f["post"]
        return BETA * (v * f["gate"] if "gate" in f else v)

    if not back:
        out, y, state = None, None, f["x"]
        if case["branch"]:
            out = ALPHA * state + added()
            state = out.float().to(t).double()
        if case["y"] == "t":
            y = _rms(state) * f["pre"]
        if case["y"] == "codes":
            # a code is by definition what 32-bit arithmetic gives
            w = state.float() * s["pre"]
            step = torch.maximum(w.abs().max(dim=1).values * torch.full((), 1 / 127, device="cuda"),
                                 torch.full((), 2.0 ** -100, device="cuda"))
            code = torch.round(w * (torch.ones_like(step) / step)[:, None]).double()
            size = torch.sqrt((state * state).sum(1) / case["n"] + EPS)
            y = code * (step.double() / size)[:, None]
        return out, y
    # the state is given: its gradient reaches the residual and the branch
    total, dpre = s["dout"].double(), None
    if case["y"]:
        normed = _rms(f["x"]) * f["pre"]
        more, dpre = torch.autograd.grad(normed, (f["x"], f["pre"]), s["dy"].double())
        total = total + more
    if not case["branch"]:
        return total, None, None, dpre, None
    names = [k for k in ("branch", "gate", "post") if k in f]
    got = dict(zip(names, torch.autograd.grad(added(), [f[k] for k in names], total)))
    return ALPHA * total, got["branch"], got.get("gate"), dpre, got.get("post")


def _exact_distill(s, case):
    losses, grads = [], []
    rows = max(1, (1 << 24) // case["v"])  # tokens at a time: bounds the 64-bit copies
    for r in range(0, case["m"], rows):
        at = slice(r, r + rows)
        logits = s["logits"][at].double().requires_grad_()
        index, t = s["index"][at].long(), s["teacher"][at].double()
        inside = index >= 0
        own_mass = torch.zeros_like(logits, requires_grad=False)
        if case["tail"]:
            p = torch.exp(t / TEMPERATURE - s["lse"][at].double()[:, None]) * inside
        else:
            p = torch.exp((t - t.max(1, keepdim=True).values) / TEMPERATURE) * inside
            p = p / p.sum(1, keepdim=True)
        own_mass = own_mass.scatter_add(1, index.clamp(min=0), p)
        logq = torch.log_softmax(logits / TEMPERATURE, dim=1)
        loss = (torch.special.xlogy(p, p)).sum(1) - (own_mass * logq).sum(1)
        if case["tail"]:
            pt = (1 - p.sum(1)).clamp(min=0)
            hit = torch.zeros_like(own_mass).scatter_add(1, index.clamp(min=0), inside.double()) > 0
            log_qt = torch.logsumexp(logq.masked_fill(hit, -math.inf), dim=1)
            loss = loss + torch.special.xlogy(pt, pt) - torch.where(pt > 0, pt * log_qt, 0)
        if s["weight"] is not None:
            loss = loss * s["weight"][at].double()
        if case["back"]:
            grads.append(torch.autograd.grad(loss, logits, s["dloss"][at].double())[0].float())
        losses.append(loss.detach())
    return (torch.cat(losses), torch.cat(grads)) if case["back"] else torch.cat(losses)


def _exact_moe(s, case):
    def codes_of(v):  # by definition what 32-bit arithmetic gives
        v = v.float()
        step = torch.maximum(v.abs().max(dim=1).values * torch.full((), 1 / 127, device="cuda"),
                             torch.full((), 2.0 ** -100, device="cuda"))
        return torch.round(v * (torch.ones_like(step) / step)[:, None]).double(), step.double()[:, None]

    fn = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
          "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
          "relu": torch.relu}[case["act"]]
    x = s["x"].double()
    scores = torch.stack([(x * row).sum(1) for row in s["router"].double()], dim=1)
    place = torch.argsort(scores, dim=1, descending=True, stable=True)[:, :case["k"]]
    soft = torch.softmax(scores, dim=1).gather(1, place)
    if case["norm"]:
        soft = torch.softmax(scores.gather(1, place), dim=1)
    q, sx = codes_of(s["x"])
    gate, gs, up, us, down, ds = s["w"]
    y = torch.zeros(case["m"], case["d"], dtype=torch.float64, device="cuda")
    for e in range(case["e"]):
        at = (place == e).nonzero()
        if not len(at):
            continue
        who = at[:, 0]
        g = q[who] @ gate[e].double().T * sx[who] * gs[e].double()
        u = q[who] @ up[e].double().T * sx[who] * us[e].double()
        qh, sh = codes_of(fn(g) * u)
        y[who] += soft[who, at[:, 1]][:, None] * (qh @ down[e].double().T * sh * ds[e].double())
    return y, None, soft


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "distill": _exact_distill, "moe": _exact_moe}[case["op"]](s, case)
