"""GPU tests of the feed-forward block on compressed Int8 weights and of the
int8 form of linear: decode, products and gradients together, against the same
operators called on the source codes (each of which has tests of its own), and
against the block in 64 bits with a bound from its two quantisations."""
import numpy as np
import pytest
import torch

import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import entropy_coded_weight_amd as E
    E.lib()
    return E


def _block(E, f, d, e, tiles=False):
    specs = [synth.random_int8_tensor(r, c, 2.0, 40 + i, c * 2) for i, (r, c) in enumerate(((f, d), (f, d), (e, f)))]
    for sp in specs:
        sp["scales"] = (np.asarray(sp["scales"], np.float32) / np.abs(sp["scales"]).max() * 0.02).astype(np.float32)
    b = E.encode_batch(specs, n_threads=4)
    p = E.plan(b.tensors, b.freq, b.chunks, b.blob.size)
    scales = torch.from_numpy(np.concatenate([sp["scales"] for sp in specs])).cuda()
    ws = []
    for sp in specs:
        codes = torch.from_numpy(np.asarray(sp["symbols"]).view(np.int8).reshape(sp["rows"], sp["cols"])).cuda()
        ws += [codes, torch.from_numpy(sp["scales"]).cuda()]
    return p, torch.from_numpy(b.blob).cuda(), scales, ws


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("m", [1, 6, 70])
def test_block_is_its_operators(E, m, kind):
    from entropy_coded_weight_amd import int8
    from entropy_coded_weight_amd.feed_forward import FeedForward
    f, d, e = 352, 256, 192
    p, blob, scales, ws = _block(E, f, d, e)
    block = FeedForward(p, scales, "gelu")
    status = torch.full((p.n_chunks,), -1, dtype=torch.int32, device="cuda")
    block.decode(blob, status)
    torch.manual_seed(m)
    x, dy = torch.randn(m, d, device="cuda").to(kind), torch.randn(m, e, device="cuda").to(kind)
    y = torch.empty(m, e, device="cuda")
    block.forward(x, y)
    assert (status == 0).all()

    h, want = torch.empty(m, f, dtype=kind, device="cuda"), torch.empty_like(y)
    int8.gated(x, None, *ws[:4], h, "gelu")
    int8.gemm(h, None, *ws[4:], want)
    assert torch.equal(y, want)

    dx, ds = torch.empty_like(x), torch.empty_like(scales)
    block.backward(dy, x, dx, ds)
    q, sx = torch.empty(m, d, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    qh, sh = torch.empty(m, f, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    int8.quantize_rows(x, q, sx)
    int8.quantize_rows(h, qh, sh)
    dh, dx2 = torch.empty_like(h), torch.empty_like(dx)
    g, u, dn = (torch.empty(n, device="cuda") for n in (f, f, e))
    int8.gemm_backward(dy, qh, sh, *ws[4:], dh, dn)
    int8.gated_backward(dh, q, sx, *ws[:4], dx2, g, u, "gelu")
    assert torch.equal(dx, dx2) and torch.equal(ds, torch.cat([g, u, dn]))

    # on a stream of the caller, with a code buffer of the caller
    side = torch.cuda.Stream()
    codes = torch.empty(p.out_elems, dtype=torch.int8, device="cuda")
    other, y2, dx3, ds3 = FeedForward(p, scales, "gelu", codes), torch.empty_like(y), torch.empty_like(dx), torch.empty_like(ds)
    torch.cuda.synchronize()
    other.decode(blob, stream=side)
    other.forward(x, y2, side)
    other.backward(dy, x, dx3, ds3, side.cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(y2, y) and torch.equal(dx3, dx) and torch.equal(ds3, ds)


def test_own_buffer_on_other_streams(E):
    """The block's own code buffer, used on a stream that is not the one it was
    allocated on, without a synchronisation by the caller: the decode waits
    for what still reads that memory, and a block that is dropped keeps it
    until its last product has run."""
    from entropy_coded_weight_amd.feed_forward import FeedForward
    f, d, e, m = 352, 256, 192, 40
    p, blob, scales, _ = _block(E, f, d, e)
    torch.manual_seed(7)
    x, dy = torch.randn(m, d, device="cuda").bfloat16(), torch.randn(m, e, device="cuda").bfloat16()
    outs = lambda: (torch.empty(m, e, device="cuda"), torch.empty_like(x), torch.empty_like(scales))  # noqa: E731
    block, want = FeedForward(p, scales), outs()
    block.decode(blob)
    block.forward(x, want[0])
    block.backward(dy, x, *want[1:])
    side = torch.cuda.Stream()
    a = torch.randn(4096, 4096, device="cuda").bfloat16()
    b = torch.empty_like(a)
    got, again = outs(), outs()

    def busy():  # some milliseconds of the current stream
        for _ in range(40):
            torch.mm(a, a, out=b)

    old = torch.full((p.out_elems,), 7, dtype=torch.int8, device="cuda")
    kept = torch.empty_like(old)
    del block
    torch.cuda.synchronize()
    busy()
    kept.copy_(old)
    del old  # its memory goes to the next allocation of this stream
    block = FeedForward(p, scales)
    block.decode(blob, stream=side)
    block.forward(x, got[0], side)
    block.backward(dy, x, *got[1:], side)
    with torch.cuda.stream(side):
        busy()
    block.forward(x, again[0], side)
    block.backward(dy, x, *again[1:], side.cuda_stream)
    del block
    junk = [torch.full((p.out_elems,), 99, dtype=torch.int8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert (kept == 7).all() and all((j == 99).all() for j in junk)
    for t in (got, again):
        assert all(torch.equal(u, v) for u, v in zip(t, want))


def test_block_in_a_graph(E):
    """Decode and both passes captured, replayed between eager calls."""
    from entropy_coded_weight_amd.feed_forward import FeedForward
    f, d, e, m = 352, 256, 192, 40
    p, blob, scales, _ = _block(E, f, d, e)
    block = FeedForward(p, scales)
    x, dy = torch.zeros(m, d, device="cuda").half(), torch.zeros(m, e, device="cuda").half()
    outs = lambda: (torch.empty(m, e, device="cuda"), torch.empty_like(x), torch.empty_like(scales))  # noqa: E731

    def step(y, dx, ds):
        block.decode(blob)
        block.forward(x, y)
        block.backward(dy, x, dx, ds)

    got = outs()
    step(*got)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*got)
    for i in range(4):
        x.copy_(torch.randn(m, d, device="cuda"))
        dy.copy_(torch.randn(m, e, device="cuda"))
        g.replay()
        want = outs()
        step(*want)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(got, want)), i


def test_block_near_the_real_numbers(E):
    """Codes are off by half a step at most: x by sx / 2 and h by sh / 2 in each
    element, which bounds what y may differ from the block in 64 bits."""
    from entropy_coded_weight_amd.feed_forward import FeedForward
    f, d, e, m = 352, 256, 192, 40
    p, blob, scales, ws = _block(E, f, d, e)
    block = FeedForward(p, scales, "relu")
    block.decode(blob)
    torch.manual_seed(5)
    x, y = torch.randn(m, d, device="cuda"), torch.empty(m, e, device="cuda")
    block.forward(x, y)
    wg, wu, wd = (ws[2 * i].double() * ws[2 * i + 1].double()[:, None] for i in range(3))
    xd = x.double()
    g, u = xd @ wg.T, xd @ wu.T
    h = g.clamp_min(0) * u
    slack = 1 + 1e-5  # fp32 arithmetic
    ex = (x.abs().amax(1, keepdim=True) / 127 / 2 * slack).double().expand_as(xd)
    eg, eu = ex @ wg.abs().T, ex @ wu.abs().T
    eh = eg * u.abs() + g.abs() * eu + eg * eu + 1e-5 * (g * u).abs()  # |relu(a) - relu(b)| <= |a - b|
    eq = ((h.abs() + eh).amax(1, keepdim=True) / 127 / 2 * slack).expand_as(h)
    bound = (eh + eq) @ wd.abs().T
    assert bool(((y.double() - h @ wd.T).abs() <= bound).all())


def test_hidden_values_beyond_float16(E):
    """float16 activations whose hidden values are not float16 numbers: a NaN
    token as stated, or with hidden_type the operators' results on fp32
    hidden values, finite and within the quantiser's step of the block in 64 bits."""
    from entropy_coded_weight_amd import int8
    from entropy_coded_weight_amd.feed_forward import FeedForward
    f, d, e, m = 352, 256, 192, 20
    p, blob, scales, ws = _block(E, f, d, e)
    torch.manual_seed(3)
    x, dy = (4000 * torch.randn(m, d, device="cuda")).half(), torch.randn(m, e, device="cuda").half()
    x[0] /= 4000
    q, sx = torch.empty(m, d, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    int8.quantize_rows(x, q, sx)
    h, want = torch.empty(m, f, device="cuda"), torch.empty(m, e, device="cuda")
    int8.gated(q, sx, *ws[:4], h, "relu")
    assert float(h.abs().amax(1)[1:].min()) > 70000 and float(h[0].abs().max()) < 60000
    qh, sh = torch.empty(m, f, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    int8.quantize_rows(h, qh, sh)
    int8.gemm(qh, sh, *ws[4:], want)
    y, narrow = torch.empty_like(want), torch.empty_like(want)
    block, plain = FeedForward(p, scales, "relu", hidden_type=torch.float32), FeedForward(p, scales, "relu")
    block.decode(blob)
    plain.decode(blob)
    block.forward(x, y)
    plain.forward(x, narrow)
    assert torch.equal(y, want) and torch.isfinite(narrow[0]).all() and torch.isnan(narrow[1:]).all()
    wd = ws[4].double() * ws[5].double()[:, None]
    bound = (0.5 * (1 + 1e-5) * h.double().abs().amax(1, keepdim=True) / 127).expand_as(h) @ wd.abs().T
    assert bool(((y.double() - h.double() @ wd.T).abs() <= bound).all())
    dx, ds, dh, dx2 = torch.empty_like(x), torch.empty_like(scales), torch.empty(m, f, device="cuda").half(), torch.empty_like(x)
    block.backward(dy, x, dx, ds)
    g, u, dn = (torch.empty(n, device="cuda") for n in (f, f, e))
    int8.gemm_backward(dy, qh, sh, *ws[4:], dh, dn)
    int8.gated_backward(dh, q, sx, *ws[:4], dx2, g, u, "relu")
    assert torch.equal(dx, dx2) and torch.equal(ds, torch.cat([g, u, dn])) and torch.isfinite(ds).all()
    with pytest.raises(E.EntqError):
        FeedForward(p, scales, hidden_type=torch.float64)


@pytest.mark.parametrize("m", [1, 90])
def test_linear_int8(E, m):
    from entropy_coded_weight_amd import int8
    from entropy_coded_weight_amd.linear import linear_int8
    p, blob, scales, ws = _block(E, 128, 256, 64)
    torch.manual_seed(m)
    xs = [torch.randn(m, int(r["cols"]), device="cuda").bfloat16() for r in p.tensors]
    ys = [torch.empty(m, int(r["rows"]), device="cuda") for r in p.tensors]
    linear_int8(p, blob, scales, xs, ys)
    for t in range(3):
        want = torch.empty_like(ys[t])
        int8.gemm(xs[t], None, ws[2 * t], ws[2 * t + 1], want)
        assert torch.equal(ys[t], want)


def _specs(f, d, e):
    specs = [synth.random_int8_tensor(r, c, 2.0, 60 + i, c * 2) for i, (r, c) in enumerate(((f, d), (f, d), (e, f)))]
    for sp in specs:
        sp["scales"] = (np.asarray(sp["scales"], np.float32) / np.abs(sp["scales"]).max() * 0.02).astype(np.float32)
    return specs


@pytest.mark.parametrize("layout,f,d,e", [("tiles", 352, 256, 192), ("tables", 512, 256, 48), ("rows", 351, 253, 191)])
def test_plans_of_every_layout(E, layout, f, d, e):
    """The block and linear_int8 on plans in tile order, with a table per chunk,
    and with matrices that start and end anywhere: the operators on the source
    codes, bit for bit."""
    from entropy_coded_weight_amd import int8
    from entropy_coded_weight_amd.feed_forward import FeedForward
    from entropy_coded_weight_amd.linear import linear_int8
    specs = _specs(f, d, e)
    if layout == "tiles":
        b = E.encode_batch([dict(sp, symbols=E.tile_order(sp["symbols"], sp["rows"], sp["cols"], 32),
                                 chunk_symbols=16 * 32, kind=sp["kind"] | E.LAYOUT_TILES) for sp in specs])
        p = E.plan(b.tensors, b.freq, b.chunks, b.blob.size)
    else:
        specs = [dict(sp, chunk_symbols=4096) for sp in specs]
        b = E.encode_batch_adaptive(specs) if layout == "tables" else E.encode_batch(specs)
        p = E.plan(b.tensors, b.freq, b.chunks, b.blob.size)
    blob, scales = torch.from_numpy(b.blob).cuda(), torch.from_numpy(np.concatenate([sp["scales"] for sp in specs])).cuda()
    ws = []
    for sp in specs:
        ws += [torch.from_numpy(np.asarray(sp["symbols"]).view(np.int8).reshape(sp["rows"], sp["cols"])).cuda(),
               torch.from_numpy(sp["scales"]).cuda()]
    torch.manual_seed(2)
    for m in (1, 40):
        x, y, want = torch.randn(m, d, device="cuda").half(), torch.empty(m, e, device="cuda"), torch.empty(m, e, device="cuda")
        block = FeedForward(p, scales, "gelu_tanh")
        block.decode(blob)
        block.forward(x, y)
        h = torch.empty(m, f, dtype=x.dtype, device="cuda")
        int8.gated(x, None, *ws[:4], h, "gelu_tanh")
        int8.gemm(h, None, *ws[4:], want)
        assert torch.equal(y, want)
        xs = [x, x, h]
        ys = [torch.empty(m, n, device="cuda") for n in (f, f, e)]
        linear_int8(p, blob, scales, xs, ys)
        for t in range(3):
            want = torch.empty_like(ys[t])
            int8.gemm(xs[t], None, ws[2 * t], ws[2 * t + 1], want)
            assert torch.equal(ys[t], want)


def test_refusals(E):
    from entropy_coded_weight_amd.feed_forward import FeedForward
    from entropy_coded_weight_amd.linear import linear_int8
    p, blob, scales, _ = _block(E, 96, 64, 32)
    bad = [lambda: FeedForward(p, scales, "swish"), lambda: FeedForward(p, scales[:-1]),
           lambda: FeedForward(p, scales, codes=torch.empty(8, dtype=torch.int8, device="cuda")),
           lambda: linear_int8(p, blob, scales, [], [])]
    q, _, s, _ = _block(E, 96, 64, 32)
    q.tensors["rows"][1] = 95
    bad.append(lambda: FeedForward(q, s))
    block = FeedForward(p, scales)
    x = torch.zeros(2, 64, device="cuda").bfloat16()
    bad += [lambda: block.forward(x[:, :63], torch.zeros(2, 32, device="cuda")),
            lambda: block.forward(x, torch.zeros(2, 31, device="cuda")),
            lambda: block.backward(torch.zeros(2, 32, device="cuda").half(), x),
            lambda: block.backward(torch.zeros(2, 32, device="cuda").bfloat16(), x, None, torch.zeros(3, device="cuda"))]
    for f in bad:
        with pytest.raises(E.EntqError) as ei:
            f()
        assert ei.value.status == E.EINVAL


def test_bad_arguments_are_refused_before_any_work(E, monkeypatch):
    """A call that refuses one of its arguments has started nothing."""
    from entropy_coded_weight_amd import feed_forward, int8, linear
    f, d, e = 96, 64, 32
    p, blob, scales, _ = _block(E, f, d, e)
    block = feed_forward.FeedForward(p, scales)
    started = []
    for module, name in ((int8, "_enqueue"), (feed_forward, "decode"), (linear, "decode")):
        monkeypatch.setattr(module, name, lambda *a, **k: started.append(a))
    new = lambda *s, t=torch.float32: torch.zeros(s, device="cuda").to(t)  # noqa: E731
    bf = torch.bfloat16
    x, y, dy = new(2, d, t=bf), new(2, e), new(2, e, t=bf)
    xs, ys = [new(2, d, t=bf), new(2, d, t=bf), new(2, f, t=bf)], [new(2, f), new(2, f), new(2, e)]
    lin = lambda xs=xs, ys=ys, **k: linear.linear_int8(p, blob, scales, xs, ys, **k)  # noqa: E731
    bad = [lambda: block.forward(x, y[:, :-1]), lambda: block.forward(x, y[:1]), lambda: block.forward(x, y.double()),
           lambda: block.forward(x, y.cpu()), lambda: block.forward(None, y), lambda: block.forward(x, None),
           lambda: block.forward(x[0], y), lambda: block.forward(x[:, :-1], y), lambda: block.forward(x.char(), y),
           lambda: block.backward(dy.float(), x.float()), lambda: block.backward(dy[:, :-1], x),
           lambda: block.backward(dy, x[:1]), lambda: block.backward(dy, x, x[:1]), lambda: block.backward(dy, x, x.half()),
           lambda: block.backward(None, x), lambda: block.backward(dy, None), lambda: block.backward(dy.half(), x),
           lambda: block.backward(dy, x, None, new(3)),
           lambda: lin(ys=ys[:2] + [new(2, e - 1)]), lambda: lin(ys=ys[:2] + [new(3, e)]),
           lambda: lin(ys=ys[:2] + [ys[2].char()]), lambda: lin(ys=ys[:2] + [None]), lambda: lin(xs=xs[:2] + [xs[2].cpu()]),
           lambda: lin(xs=xs[:2] + [xs[2][:, :-1]]), lambda: lin(xs=xs[:2] + [xs[2].char()]),
           lambda: lin(codes=new(p.out_elems, t=torch.uint8)), lambda: lin(codes=new(p.out_elems - 1, t=torch.int8))]
    for i, call in enumerate(bad):
        with pytest.raises(E.EntqError) as ei:
            call()
        assert ei.value.status == E.EINVAL and not started, i
    lin()
    block.forward(x, y)
    block.backward(dy, x, torch.empty_like(x), torch.empty_like(scales))
    assert len(started) == 4 + 2 + 5


def test_buffers_of_any_shape(E):
    """Code and scale buffers are taken by their elements, whatever their shape."""
    from entropy_coded_weight_amd import int8
    from entropy_coded_weight_amd.feed_forward import FeedForward
    from entropy_coded_weight_amd.linear import linear_int8
    f, d, e = 96, 64, 32
    p, blob, scales, ws = _block(E, f, d, e)
    codes = torch.empty(p.out_elems // 32, 32, dtype=torch.int8, device="cuda")
    x, y, want = torch.randn(3, d, device="cuda").bfloat16(), torch.empty(3, e, device="cuda"), torch.empty(3, e, device="cuda")
    plain = FeedForward(p, scales)
    plain.decode(blob)
    plain.forward(x, want)
    block = FeedForward(p, scales.view(-1, 2), codes=codes)
    block.decode(blob)
    block.forward(x, y)
    assert torch.equal(y, want)
    dy = torch.randn(3, e, device="cuda").bfloat16()
    a, b = torch.zeros(p.scale_rows, device="cuda"), torch.zeros(p.scale_rows // 2, 2, device="cuda")
    plain.backward(dy, x, None, a)
    block.backward(dy, x, None, b)
    assert torch.equal(a, b.view(-1)) and bool((a != 0).any())
    xs = [x, x, torch.randn(3, f, device="cuda").bfloat16()]
    for c in (None, codes):
        ys = [torch.empty(3, n, device="cuda") for n in (f, f, e)]
        linear_int8(p, blob, scales.view(2, -1), xs, ys, codes=c)
        for t in range(3):
            want = torch.empty_like(ys[t])
            int8.gemm(xs[t], None, ws[2 * t], ws[2 * t + 1], want)
            assert torch.equal(ys[t], want)


def test_autograd(E):
    """Activations that need a graph are refused, and a function around the two
    calls gives their gradients, the scales' among them."""
    from entropy_coded_weight_amd import int8, linear
    from entropy_coded_weight_amd.feed_forward import FeedForward
    f, d, e, m = 96, 64, 32, 5
    p, blob, scales, ws = _block(E, f, d, e)
    scales.requires_grad_(True)
    block = FeedForward(p, scales, "silu")
    block.decode(blob)

    class Block(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, scales):
            ctx.save_for_backward(x)
            y = torch.empty(m, e, dtype=x.dtype, device="cuda")
            block.forward(x, y)
            return y

        @staticmethod
        def backward(ctx, dy):
            dx, ds = torch.empty_like(ctx.saved_tensors[0]), torch.empty_like(scales)
            block.backward(dy.contiguous(), ctx.saved_tensors[0], dx, ds)
            return dx, ds

    torch.manual_seed(1)
    x = torch.randn(m, d, device="cuda").bfloat16().requires_grad_(True)
    dy = torch.randn(m, e, device="cuda").bfloat16()
    Block.apply(x, scales).backward(dy)
    dx, ds = torch.empty_like(x), torch.empty_like(scales)
    block.backward(dy, x.detach(), dx, ds)
    assert torch.equal(x.grad, dx) and torch.equal(scales.grad, ds) and bool((ds != 0).any())

    y, h = torch.empty(m, e, device="cuda"), torch.empty(m, f, device="cuda")
    q, sx = torch.empty(m, d, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    dh = torch.zeros(m, f, device="cuda").half().requires_grad_(True)
    calls = [lambda: block.forward(x, y), lambda: block.backward(dy, x), lambda: int8.quantize_rows(x, q, sx),
             lambda: int8.gemm(x, None, *ws[:2], h), lambda: int8.gated(x, None, *ws[:4], h),
             lambda: int8.gemm_backward(dh, q, sx, *ws[:2]), lambda: int8.gated_backward(dh, q, sx, *ws[:4]),
             lambda: linear.linear_int8(p, blob, scales, [x, x, h.bfloat16()], [h, h.clone(), y])]
    for call in calls:
        with pytest.raises(E.EntqError, match="requires a gradient") as ei:
            call()
        assert ei.value.status == E.EINVAL
    with torch.no_grad():
        for call in calls:
            call()
