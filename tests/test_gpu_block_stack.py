"""GPU tests of what the operators around a block are used for: a residual
block between its norms, the distillation of a compressed output projection,
and a run of all of them together."""
import numpy as np
import pytest
import torch

import distill_reference
import int8_reference
import synth
from int8_reference import EPS
from norm_reference import TYPES, rho

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import entropy_coded_weight_amd as E
    E.lib()
    return E


def plan_of(E, shapes, seed=40):
    """plan, container, scales and the source codes with their scales"""
    specs = [synth.random_int8_tensor(r, c, 2.0, seed + i, 4096) for i, (r, c) in enumerate(shapes)]
    for sp in specs:
        sp["scales"] = (np.asarray(sp["scales"], np.float32) / np.abs(sp["scales"]).max() * 0.02).astype(np.float32)
    b = E.encode_batch(specs, n_threads=4)
    p = E.plan(b.tensors, b.freq, b.chunks, b.blob.size)
    scales = torch.from_numpy(np.concatenate([sp["scales"] for sp in specs])).cuda()
    ws = []
    for sp in specs:
        ws += [torch.from_numpy(np.asarray(sp["symbols"]).view(np.int8).reshape(sp["rows"], sp["cols"])).cuda(),
               torch.from_numpy(sp["scales"]).cuda()]
    return p, torch.from_numpy(b.blob).cuda(), scales, ws


def vector(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 1 + 0.3 * torch.randn(n, device="cuda", generator=g)


def gates(which, m, d, kind):
    torch.manual_seed(11)
    return {"none": None, "channel": vector(d, 9), "token": torch.randn(m, 1, device="cuda"),
            "full": torch.randn(m, d, device="cuda").to(TYPES[kind])}[which]


def residual_setup(E, m, d, f, kind):
    from entropy_coded_weight_amd.feed_forward import FeedForward
    p, blob, scales, ws = plan_of(E, ((f, d), (f, d), (d, f)))
    block = FeedForward(p, scales, "gelu")
    block.decode(blob)
    torch.manual_seed(m)
    return block, ws, scales, torch.randn(m, d, device="cuda").to(TYPES[kind])


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("m,d,f,kind", [(1, 256, 352, "bf16"), (37, 253, 351, "f16"), (70, 256, 352, "f32")])
def test_residual_is_its_operators(E, m, d, f, kind, gate, post):
    from entropy_coded_weight_amd import int8, norm
    block, ws, scales, x = residual_setup(E, m, d, f, kind)
    pre, w, g = vector(d, 1), vector(d, 2) if post else None, gates(gate, m, d, kind)
    out = torch.empty_like(x)
    block.residual(x, out, pre, w, g, 0.5, 1.25, 1e-5)
    q, sx = torch.empty(m, d, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    norm.block(x, pre=pre, y=q, y_scales=sx, eps=1e-5)
    h, y, want = torch.empty(m, f, dtype=x.dtype, device="cuda"), torch.empty_like(x), torch.empty_like(x)
    int8.gated(q, sx, *ws[:4], h, "gelu")
    int8.gemm(h, None, *ws[4:], y)
    norm.block(x, y, want, w, g, alpha=0.5, beta=1.25, eps=1e-5)
    assert torch.equal(out, want) and bool((out != x).any())
    own = x.clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    block.residual(own, own, pre, w, g, 0.5, 1.25, 1e-5, side)
    torch.cuda.synchronize()
    assert torch.equal(own, out)


@pytest.mark.parametrize("alpha,gate,post", [(1.0, "none", False), (1.0, "channel", True), (0.5, "token", True),
                                             (1.0, "full", False), (-0.5, "full", True)])
@pytest.mark.parametrize("m,d,f", [(1, 256, 352), (37, 253, 351)])
def test_residual_gradients(E, m, d, f, alpha, gate, post):
    """Against autograd in 64 bits with the quantisers passed straight through.
    Six roundings to float16 stand one after the other (y, dy, dh, each product's
    scaled gradient twice, dn, the result), each at most 2^-11 of its values; twice
    their sum is allowed of a gradient's Frobenius norm, since a map may
    take less from the gradient than from a rounding's error."""
    from entropy_coded_weight_amd import int8, norm
    block, ws, scales, x = residual_setup(E, m, d, f, "f16")
    pre, w, g = vector(d, 1), vector(d, 2) if post else None, gates(gate, m, d, "f16")
    dout = torch.randn(m, d, device="cuda").half()
    got = {"dx": torch.empty_like(x), "dscales": torch.empty_like(scales), "dpre": torch.empty(d, device="cuda")}
    if post:
        got["dpost"] = torch.empty(d, device="cuda")
    if g is not None:
        got["dgate"] = torch.empty_like(g)
    call = lambda **k: block.residual_backward(dout, x, pre, w, g, alpha=alpha, beta=1.25, eps=1e-5, **k)  # noqa: E731
    call(**got)
    q, sx = torch.empty(m, d, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    norm.block(x, pre=pre, y=q, y_scales=sx, eps=1e-5)
    h = torch.empty(m, f, dtype=x.dtype, device="cuda")
    int8.gated(q, sx, *ws[:4], h, "gelu")
    qh, sh = torch.empty(m, f, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    int8.quantize_rows(h, qh, sh)

    leaf = {"dx": x.double(), "dscales": scales.double(), "dpre": pre.double(), "dpost": w.double() if post else None,
            "dgate": g.double() if g is not None else None}
    for t in leaf.values():
        if t is not None:
            t.requires_grad_()
    sg, su, sd = leaf["dscales"][:f], leaf["dscales"][f:2 * f], leaf["dscales"][2 * f:]
    straight = lambda v, to: v + (to - v).detach()  # noqa: E731
    n = straight(leaf["dx"] * rho(leaf["dx"], 1e-5) * leaf["dpre"], q.double() * sx.double()[:, None])
    a = n @ ws[0].double().T * sg
    hidden = 0.5 * a * torch.erfc(-a / 2 ** 0.5) * (n @ ws[2].double().T * su)
    y = straight(hidden, qh.double() * sh.double()[:, None]) @ ws[4].double().T * sd
    v = y * rho(y, 1e-5) * leaf["dpost"] if post else y
    out = alpha * leaf["dx"] + 1.25 * (leaf["dgate"] if g is not None else 1) * v
    out.backward(dout.double())
    for name, t in got.items():
        want = leaf[name].grad
        assert float((t.double() - want).norm()) <= 2 * 6 * 2.0 ** -11 * float(want.norm()), name
        alone = torch.empty_like(t)
        call(**{name: alone})
        assert torch.equal(alone, t), name


def test_residual_of_no_tokens(E):
    block, _, scales, _ = residual_setup(E, 1, 256, 352, "f16")
    x, pre, post = torch.empty(0, 256, device="cuda").half(), vector(256, 1), vector(256, 2)
    block.residual(x, x.clone(), pre, post, vector(256, 3))
    got = [torch.ones_like(scales)] + [torch.ones(256, device="cuda") for _ in range(3)]
    block.residual_backward(x, x, pre, post, vector(256, 3), x.clone(), *got)
    assert not any(bool(t.any()) for t in got)


def head_inputs(m, v, d, k, kind, tail, seed=3):
    torch.manual_seed(seed)
    x = torch.randn(m, d, device="cuda").to(TYPES[kind])
    teacher = 3 * torch.randn(m, v, device="cuda")
    top, index = torch.topk(teacher, k, dim=1)
    weight = torch.rand(m, device="cuda") + 0.25
    weight[:m - 1:5] = 0
    return x, index.int(), top, torch.logsumexp(teacher / 1.25, 1) if tail else None, weight


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("m,v,d,k,kind,tokens", [(1, 1000, 256, 8, "bf16", 1024), (70, 1000, 256, 20, "f16", 32),
                                                (33, 5003, 130, 64, "bf16", 16)])
def test_distillation_of_a_projection(E, m, v, d, k, kind, tokens, tail):
    from entropy_coded_weight_amd import int8
    from entropy_coded_weight_amd.linear import distill_int8
    p, blob, scales, (w, ws) = plan_of(E, ((v, d),))
    x, index, top, lse, weight = head_inputs(m, v, d, k, kind, tail)
    x[:m - 1:5] = float("nan")  # tokens of weight 0: no loss, no gradient, no trace in dscales
    dloss = torch.rand(m, device="cuda")
    loss, dx, ds = torch.full((m,), 7.0, device="cuda"), torch.empty_like(x), torch.full((v,), 7.0, device="cuda")
    rest = dict(dloss=dloss, teacher_lse=lse, weight=weight, temperature=1.25, tokens=tokens)
    distill_int8(p, blob, scales, x, index, top, loss, dx, ds, **rest)
    q, sx = torch.empty(m, d, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    z = torch.empty(m, v, device="cuda")
    int8.quantize_rows(x, q, sx)
    int8.gemm(q, sx, w, ws, z)
    (want, bound), (g, gb) = distill_reference.distill(z, index, top, lse, weight, 1.25, dloss, kind)
    assert ((loss.double() - want).abs() <= bound).all()
    (rx, bx), _ = int8_reference.gemm_backward(g, q, sx, w, ws, kind)
    s = ws.double()
    bx = bx + (gb * s) @ w.double().abs() * (1 + int8_reference.ROUND[kind])
    assert ((dx.double() - rx).abs() <= bx).all() and bool((dx[:m - 1:5] == 0).all())
    z = int8_reference.sums(q, w) * sx.nan_to_num(0).double()[:, None]
    t = g * z
    # (a group's sum in fp32, then the groups')
    b = (m + 8 + m // tokens + 1) * EPS * t.abs().sum(0) + 1.001 * (gb * z.abs()).sum(0)
    assert ((ds.double() - t.sum(0)).abs() <= b).all() and bool((ds != 0).any())
    # each alone, the losses alone, and on a stream with codes of the caller
    for name, t in (("dx", dx), ("dscales", ds)):
        other, again = torch.empty_like(loss), torch.empty_like(t)
        distill_int8(p, blob, scales, x, index, top, other, **{name: again}, **rest)
        assert torch.equal(again, t) and torch.equal(other, loss)
    other = torch.empty_like(loss)
    distill_int8(p, blob, scales, x, index, top, other, **rest)
    assert ((other.double() - want).abs() <= bound).all()
    codes, side = torch.empty(p.out_elems, dtype=torch.int8, device="cuda"), torch.cuda.Stream()
    status = torch.full((p.n_chunks,), -1, dtype=torch.int32, device="cuda")
    dx2, ds2 = torch.empty_like(dx), torch.empty_like(ds)
    torch.cuda.synchronize()
    distill_int8(p, blob, scales, x, index, top, other, dx2, ds2, codes=codes, chunk_status=status, stream=side, **rest)
    torch.cuda.synchronize()
    assert torch.equal(dx2, dx) and torch.equal(ds2, ds) and torch.equal(other, loss) and bool((status == 0).all())


def test_distillation_of_no_tokens(E):
    from entropy_coded_weight_amd.linear import distill_int8
    p, blob, scales, _ = plan_of(E, ((40, 24),))
    new = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    ds = new(40)
    distill_int8(p, blob, scales, new(0, 24).half(), torch.zeros(0, 3, dtype=torch.int32, device="cuda"), new(0, 3), new(0),
                 new(0, 24).half(), ds)
    assert not ds.any()


def test_all_together(E):
    """A residual block, a mixture of experts on the normed state, and the
    distillation of the head, forward and backward, eager and captured; the
    router's norm feeds the mixture in the state's type."""
    from entropy_coded_weight_amd import norm
    from entropy_coded_weight_amd.feed_forward import FeedForward
    from entropy_coded_weight_amd.linear import distill_int8
    from entropy_coded_weight_amd.moe import MixtureOfExperts
    d, f, v, e, m, k = 192, 352, 700, 3, 21, 12
    p, blob, scales, _ = plan_of(E, ((f, d), (f, d), (d, f)))
    pe, blobe, scalese, _ = plan_of(E, [s for _ in range(e) for s in ((64, d), (64, d), (d, 64))], 70)
    ph, blobh, scalesh, _ = plan_of(E, ((v, d),), 90)
    torch.manual_seed(8)
    router = torch.randn(e, d, device="cuda")
    block, experts = FeedForward(p, scales), MixtureOfExperts(pe, scalese, router, 2)
    pre, post, pre2, last = (vector(d, i) for i in range(4))
    x, index, top, lse, weight = head_inputs(m, v, d, k, "bf16", True)
    bf = lambda: torch.empty(m, d, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    fl = lambda n: torch.empty(n, device="cuda")  # noqa: E731

    def outs():
        return {"loss": fl(m), "state": bf(), "state2": bf(), "final": bf(), "moe": bf(), "normed": bf(), "dx": bf(),
                "dfinal": bf(), "dhead": fl(v), "dstate2": bf(), "dlast": fl(d), "dscales": torch.empty_like(scales), "dpre": fl(d),
                "dpost": fl(d)}

    def step(o):
        block.decode(blob)
        experts.decode(blobe)
        block.residual(x, o["state"], pre, post)
        norm.block(o["state"], pre=pre2, y=o["normed"])
        experts.forward(o["normed"], o["moe"])
        norm.block(o["state"], o["moe"], o["state2"], pre=last, y=o["final"])
        distill_int8(ph, blobh, scalesh, o["final"], index, top, o["loss"], o["dfinal"], o["dhead"], teacher_lse=lse, weight=weight,
                     temperature=1.25, tokens=8)
        norm.block_backward(o["state2"], dy=o["dfinal"], pre=last, dx=o["dstate2"], dpre=o["dlast"])
        # (of the block below as if the mixture were constant)
        block.residual_backward(o["dstate2"], x, pre, post, dx=o["dx"], dscales=o["dscales"], dpre=o["dpre"], dpost=o["dpost"])

    got = outs()
    step(got)
    torch.cuda.synchronize()
    assert all(bool(torch.isfinite(t).all()) and bool(t.any()) for t in got.values())
    # a step along the negative gradient of the head's scales lowers the loss as they say
    lower = fl(m)
    sign = got["dhead"].sign()
    by = 1e-3 * scalesh * sign
    distill_int8(ph, blobh, scalesh - by, got["final"], index, top, lower, teacher_lse=lse, weight=weight, temperature=1.25)
    higher = fl(m)
    distill_int8(ph, blobh, scalesh + by, got["final"], index, top, higher, teacher_lse=lse, weight=weight, temperature=1.25)
    change, said = float((higher - lower).double().sum()), 2 * float((by.double() * got["dhead"].double()).sum())
    # bf16 logits' gradients: 2^-8 of each term, terms of both signs; 5 %
    assert abs(change - said) <= 0.05 * said
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(got)
    for i in range(3):
        x.copy_(torch.randn(m, d, device="cuda"))
        graph.replay()
        want = outs()
        step(want)
        torch.cuda.synchronize()
        for name, t in want.items():
            assert torch.equal(t, got[name]), (i, name)


def test_refusals(E, monkeypatch):
    """A call that refuses one of its arguments has started nothing."""
    from entropy_coded_weight_amd import feed_forward, int8, linear, norm
    d, f, v, m = 64, 96, 40, 3
    p, blob, scales, _ = plan_of(E, ((f, d), (f, d), (d, f)))
    ph, blobh, scalesh, _ = plan_of(E, ((v, d),))
    pn, _, scalesn, _ = plan_of(E, ((f, d), (f, d), (32, f)))
    block, narrow = feed_forward.FeedForward(p, scales), feed_forward.FeedForward(pn, scalesn)
    started = []
    for module, name in ((int8, "_enqueue"), (norm, "_enqueue"), (linear, "decode")):
        monkeypatch.setattr(module, name, lambda *a, **k: started.append(a))
    new = lambda *s, t=torch.float32: torch.ones(s, device="cuda").to(t)  # noqa: E731
    bf = torch.bfloat16
    x, o, w, g = new(m, d, t=bf), new(m, d, t=bf), new(d), new(m, 1)
    leaf = x.clone().requires_grad_()
    R, B = block.residual, block.residual_backward
    index, top, loss = torch.zeros(m, 4, dtype=torch.int32, device="cuda"), new(m, 4), new(m)
    H = lambda x=x, index=index, top=top, loss=loss, plan=ph, s=scalesh, **k: linear.distill_int8(  # noqa: E731
        plan, blobh, s, x, index, top, loss, **k)
    bad = [lambda: R(x, o, None), lambda: R(x, o.half(), w), lambda: R(x, o[:2], w), lambda: R(x, o, w[:9]), lambda: R(x.char(), o, w),
           lambda: R(x[:, :9], o[:, :9], w[:9]), lambda: R(x, o, w, w.half()), lambda: R(x, o, w, gate=new(m, d)),
           lambda: R(x, o, w, eps=0.0), lambda: R(x, o, w, alpha=float("inf")), lambda: R(leaf, o, w), lambda: R(x, None, w),
           lambda: narrow.residual(x, o, w), lambda: R(x.cpu(), o, w), lambda: R(None, o, w),
           lambda: B(o, x, None), lambda: B(o.half(), x, w), lambda: B(o.float(), x.float(), w), lambda: B(o[:2], x, w),
           lambda: B(leaf, x, w), lambda: B(o, leaf, w), lambda: B(o, x, w, dx=x.half()), lambda: B(o, x, w, dpost=w),
           lambda: B(o, x, w, dgate=w), lambda: B(o, x, w, gate=g, dgate=w), lambda: B(o, x, w, dpre=w[:3]),
           lambda: B(o, x, w, dscales=w[:3]), lambda: B(None, x, w), lambda: narrow.residual_backward(o, x, w),
           lambda: H(x.float()), lambda: H(x[:, :9]), lambda: H(leaf), lambda: H(index=index[:2]), lambda: H(index=index.short()),
           lambda: H(top=top[:2]), lambda: H(top=top.double()), lambda: H(top=top[:, :0], index=index[:, :0]), lambda: H(loss=loss[:2]),
           lambda: H(loss=None), lambda: H(dx=x.half()), lambda: H(dscales=w[:9]), lambda: H(dloss=loss[:2]),
           lambda: H(weight=loss[:2]), lambda: H(teacher_lse=loss[:2]), lambda: H(temperature=0), lambda: H(tokens=0),
           lambda: H(tokens=1.5), lambda: H(plan=p, s=scales), lambda: H(codes=new(8, t=torch.int8)), lambda: H(index=None),
           lambda: H(top=None), lambda: H(x=None)]
    for i, call in enumerate(bad):
        with pytest.raises(E.EntqError) as ei:
            call()
        assert ei.value.status == E.EINVAL and not started, i
