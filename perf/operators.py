"""The int8 operators measured: the product of quantised activations with
int8 weight codes (a scale per token and per channel), the gated feed-forward
kernel on such codes, and the backward pass of each.

A case's fields: op ("product" or "gated"), back (the backward pass), m
tokens, n channels, k columns of the weights, x (the activations' type, or in
a backward pass the gradients' type), out (the result's type, forward only),
act (the gated operator's activation)."""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def _product(name, m, n, k, x, out):
    return {"name": name, "op": "product", "back": False, "m": m, "n": n, "k": k, "x": x,
            "out": out}


def _gated(name, m, n, k, x, out, act):
    return {"name": name, "op": "gated", "back": False, "m": m, "n": n, "k": k, "x": x,
            "out": out, "act": act}


def listed():
    return [
        # one generated token through a square projection: latency and one read of the weights
        _product("product_token", 1, 8192, 8192, "bf16", "bf16"),
        # a few sequences' keys or values (8 shared heads of 128), fp32 in and out: the smallest call
        _product("product_kv_few", 7, 1024, 8192, "f32", "f32"),
        # the logits of 16 sequences: the longest list of channels
        _product("product_lm_head", 16, 32000, 8192, "bf16", "f32"),
        # a short prompt with odd sides: every row of the weights starts at another alignment
        _product("product_ragged", 333, 5121, 4099, "f16", "f16"),
        # the down projection of a long prompt
        _product("product_prefill", 4096, 8192, 28672, "bf16", "bf16"),
        # gradients through a key projection for a short sequence
        {"name": "product_back_short", "op": "product", "back": True, "m": 96, "n": 1024,
         "k": 8192, "x": "f16"},
        # gradients through a square projection for one training batch of tokens
        {"name": "product_back", "op": "product", "back": True, "m": 2048, "n": 8192, "k": 8192,
         "x": "bf16"},
        # one generated token through gate and up
        _gated("gated_token", 1, 28672, 8192, "bf16", "bf16", "silu"),
        # 48 sequences in step, the smaller block
        _gated("gated_batch", 48, 13824, 5120, "f16", "f16", "gelu_tanh"),
        # a long prompt through gate and up: the largest case
        _gated("gated_prefill", 4096, 28672, 8192, "bf16", "bf16", "silu"),
        # a small model with odd sides, in training
        {"name": "gated_back_ragged", "op": "gated", "back": True, "m": 515, "n": 2753,
         "k": 1031, "x": "bf16", "act": "gelu"},
        # the large block in training
        {"name": "gated_back", "op": "gated", "back": True, "m": 2048, "n": 28672, "k": 8192,
         "x": "bf16", "act": "silu"},
    ]


def draw(rng):
    while True:
        def side(lo, hi):
            v = round(math.exp(rng.uniform(math.log(lo), math.log(hi))))
            step = rng.choice((64, 64, 16, 1))
            return max(step, v // step * step)
        c = {"op": rng.choice(("product", "gated")), "back": rng.random() < 0.4,
             "m": round(math.exp(rng.uniform(0.0, math.log(4096)))),
             "n": side(256, 32000), "k": side(256, 28672)}
        if c["back"]:
            c["x"] = rng.choice(("bf16", "f16"))
        else:
            c["x"] = rng.choice(("bf16", "bf16", "f16", "f32"))
            c["out"] = rng.choice((c["x"], "f32"))
        if c["op"] == "gated":
            c["act"] = rng.choice(ACTS)
        w = work(c)
        if w["flops"] <= 2e12 and w["bytes"] <= 6e8:
            return c


def work(case):
    m, n, k = case["m"], case["n"], case["k"]
    weights = 2 if case["op"] == "gated" else 1
    e = BYTES[case["x"]]
    if case["back"]:
        # gradient and codes in, dX and the scales' gradients out
        return {"bytes": m * n * e + m * k + 4 * m + weights * (n * k + 8 * n) + m * k * e,
                "flops": 4 * weights * m * n * k}
    return {"bytes": m * k * e + weights * (n * k + 4 * n) + m * n * BYTES[case["out"]],
            "flops": 2 * weights * m * n * k}


def _weights(n, k, g):
    """Codes as a weight quantiser leaves them (Laplacian, a few bits of
    entropy) and a positive scale per row."""
    codes = torch.empty(n, k, dtype=torch.int8, device="cuda")
    for r in range(0, n, 4096):
        e = torch.empty(min(4096, n - r), k, device="cuda").exponential_(1.0, generator=g)
        s = torch.rand(e.shape, device="cuda", generator=g)
        codes[r:r + e.shape[0]] = (torch.where(s < 0.5, -e, e) * 2.0).round().clamp(-127, 127)
    scales = 0.007 * torch.exp(0.3 * torch.randn(n, device="cuda", generator=g))
    return codes, scales


def _activations(m, k, g):
    """Hidden states: normal, with channels of very different size and a few
    that stand far out."""
    size = torch.exp(0.5 * torch.randn(k, device="cuda", generator=g))
    size[torch.rand(k, device="cuda", generator=g) < 0.002] *= 10
    return torch.randn(m, k, device="cuda", generator=g) * size


def _quantise(x):
    """Codes and scales of the rows of x, in 32 bits."""
    x = x.float()
    scale = (x.abs().amax(1) * torch.tensor(1 / 127, dtype=torch.float32)).clamp_min(2.0 ** -100)
    inv = torch.reciprocal(scale)
    return (x * inv[:, None]).round().clamp(-127, 127), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    m, n, k = case["m"], case["n"], case["k"]
    s = {"case": case, "w": [_weights(n, k, g) for _ in range(2 if case["op"] == "gated" else 1)]}
    x = _activations(m, k, g)
    new = lambda *shape, dtype: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if case["back"]:
        t = TYPES[case["x"]]
        q, s["sx"] = _quantise(x)
        s["q"] = q.to(torch.int8)
        # fp16 training scales its loss, bf16 training does not
        dy = torch.randn(m, n, device="cuda", generator=g) * (1.0 if case["x"] == "f16" else 1e-3)
        s["dy"] = dy.to(t)
        s["dx"] = new(m, k, dtype=t)
        s["ds"] = [new(n, dtype=torch.float32) for _ in s["w"]]
    else:
        s["x"] = x.to(TYPES[case["x"]])
        s["y"] = new(m, n, dtype=TYPES[case["out"]])
    return s


def _act(name, v):
    """act(v) and act'(v)."""
    if name == "silu":
        p = 1 / (1 + torch.exp(-v))
        return v * p, p * (1 + v * (1 - p))
    if name == "gelu":
        p = 0.5 * (1 + torch.erf(v * math.sqrt(0.5)))
        return v * p, p + v * torch.exp(-0.5 * v * v) * (1 / math.sqrt(2 * math.pi))
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (v + 0.044715 * v * v * v))
        return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * c * (1 + 0.134145 * v * v)
    return torch.where(v > 0, v, 0), (v > 0).to(v.dtype)


def _plain(s):
    case = s["case"]
    w = [c.float() for c, _ in s["w"]]
    scales = [sc for _, sc in s["w"]]
    if case["back"]:
        q, sx = s["q"].float(), s["sx"]
    else:
        q, sx = _quantise(s["x"])
    acc = [torch.mm(q, v.t()) * sx[:, None] for v in w]  # without the channel's scale
    if not case["back"]:
        out = TYPES[case["out"]]
        if case["op"] == "product":
            return (acc[0] * scales[0]).to(out)
        return (_act(case["act"], acc[0] * scales[0])[0] * (acc[1] * scales[1])).to(out)
    d = [s["dy"].float()]
    if case["op"] == "gated":
        a, da = _act(case["act"], acc[0] * scales[0])
        d = [d[0] * (acc[1] * scales[1]) * da, d[0] * a]
    dx = torch.mm(d[0] * scales[0], w[0])
    if case["op"] == "gated":
        dx += torch.mm(d[1] * scales[1], w[1])
    return dx.to(s["dy"].dtype), [(v * t).sum(0) for v, t in zip(d, acc)]


def _own(s):
    from entropy_coded_weight_amd import int8
    case, w = s["case"], s["w"]
    if case["op"] == "product":
        if not case["back"]:
            int8.gemm(s["x"], None, *w[0], s["y"])
            return s["y"]
        int8.gemm_backward(s["dy"], s["q"], s["sx"], *w[0], s["dx"], s["ds"][0])
    else:
        if not case["back"]:
            int8.gated(s["x"], None, *w[0], *w[1], s["y"], case["act"])
            return s["y"]
        int8.gated_backward(s["dy"], s["q"], s["sx"], *w[0], *w[1], s["dx"], *s["ds"],
                            case["act"])
    return s["dx"], s["ds"]


def run(state):
    return _own(state) if own else _plain(state)


def exact(case, seed):
    s = prepare(case, seed)
    rows = max(1, (1 << 28) // max(case["n"], case["k"]))  # tokens at a time: bounds the 64-bit copies
    weights = [(c.double(), sc.double()) for c, sc in s["w"]]
    outs, sums = [], [0.0 for _ in weights]
    for r in range(0, case["m"], rows):
        if case["back"]:
            code, step = s["q"][r:r + rows].double(), s["sx"][r:r + rows]
        else:
            # a code is by definition what 32-bit arithmetic gives
            x = s["x"][r:r + rows].to(torch.float32)
            step = torch.maximum(x.abs().max(dim=1).values * torch.full((), 1 / 127, device="cuda"),
                                 torch.full((), 2.0 ** -100, device="cuda"))
            code = torch.round(x * (torch.ones_like(step) / step).unsqueeze(1)).double()
        raw = [(code @ v.T) * step.double().unsqueeze(1) for v, _ in weights]
        z = [a * sc for a, (_, sc) in zip(raw, weights)]
        if case["op"] == "gated":
            g = z[0].requires_grad_(case["back"])
            name = case["act"]
            f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
                 "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh"),
                 "relu": torch.relu}[name](g)
        if not case["back"]:
            outs.append(f * z[1] if case["op"] == "gated" else z[0])
            continue
        dy = s["dy"][r:r + rows].double()
        d = [dy]
        if case["op"] == "gated":
            d = [torch.autograd.grad(f, g, dy * z[1])[0], dy * f.detach()]
        outs.append(sum((v * sc) @ wt for v, (wt, sc) in zip(d, weights)))
        sums = [t + (v * a.detach()).sum(dim=0) for t, v, a in zip(sums, d, raw)]
    y = torch.cat(outs).detach()
    return (y, sums) if case["back"] else y
