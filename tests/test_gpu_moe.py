"""GPU tests of the mixture-of-experts layer on int8 codes against a 64-bit
reference, and of the layer on a plan."""
import numpy as np
import pytest
import torch

import moe_reference as R
import synth
from int8_reference import EPS
from norm_reference import TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import entropy_coded_weight_amd as E
    E.lib()
    return E


@pytest.fixture(scope="module")
def M(E):
    from entropy_coded_weight_amd import moe
    return moe


def codes(e, r, c, g, pad=0):
    """[e, r, c] codes; pad: bytes between the rows, so that they start anywhere"""
    v = torch.randint(-127, 128, (e, r, c + pad), device="cuda", generator=g, dtype=torch.int8)
    v = torch.where(torch.rand(v.shape, device="cuda", generator=g) < 0.9, v // 24, v)
    return v[:, :, pad // 2:pad // 2 + c]


def layer(m, e, d, f, n, kind, router_kind, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(m, d + pad, device="cuda", generator=g).to(TYPES[kind])[:, :d]
    router = (torch.randn(e, d + pad, device="cuda", generator=g) * (2 / d ** 0.5)).to(TYPES[router_kind])[:, :d]
    s = lambda r, c: (0.3 / c ** 0.5) * (0.5 + torch.rand(e, r + pad, device="cuda", generator=g))[:, :r]  # noqa: E731
    return x, router, [codes(e, f, d, g, pad), s(f, d), codes(e, f, d, g, pad), s(f, d), codes(e, n, f, g, pad), s(n, f)]


def check(M, x, router, w, k, act, normalize, kind, workspace=None):
    m, n = x.shape[0], w[4].shape[1]
    flat = torch.full((m, n + 5), 7.0, device="cuda").to(TYPES[kind])
    y = flat[:, 2:n + 2]
    experts = torch.full((m, k), -9, dtype=torch.int32, device="cuda")
    p = torch.full((m, k), -9.0, device="cuda")
    M.few(x, router, *w, y, k, act, normalize, experts, p, workspace=workspace)
    at, want_p, want, bound = R.layer(x, router, *w, k, act, normalize, kind)
    assert torch.equal(experts.long(), at)
    assert ((p.double() - want_p).abs() <= 4 * EPS * want_p).all()
    bad = ~((y.double() - want).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), float((y.double() - want).abs().max()), float(bound.max()))
    assert bool((flat[:, :2] == 7).all()) and bool((flat[:, n + 2:] == 7).all())
    # y alone, over a workspace of other bytes
    again = torch.empty(m, n, dtype=y.dtype, device="cuda")
    room = M.workspace_bytes(x, router, *w, k)
    M.few(x, router, *w, again, k, act, normalize, workspace=torch.full((room,), 0xA5, dtype=torch.uint8, device="cuda"))
    assert torch.equal(again, y)
    return y


SIZES = [(1, 8, 2, 256, 352, 192), (1, 1, 1, 16, 16, 16), (1, 64, 6, 512, 128, 260), (2, 3, 3, 1, 1, 1), (3, 5, 5, 130, 77, 33),
         (5, 60, 4, 1100, 700, 500), (8, 128, 8, 384, 96, 144), (16, 16, 4, 640, 1030, 128), (17, 9, 2, 200, 129, 70),
         (33, 64, 6, 256, 160, 96), (48, 256, 32, 130, 64, 40), (64, 4, 1, 1024, 512, 300), (64, 200, 8, 96, 48, 32),
         (1, 4, 2, 2048, 5000, 96), (4, 2, 2, 70, 40000, 20)]


@pytest.mark.parametrize("kind,router_kind,act,normalize", [("bf16", "f32", "silu", True), ("f16", "f16", "gelu", False),
                                                            ("f32", "bf16", "gelu_tanh", True), ("bf16", "bf16", "relu", False)])
@pytest.mark.parametrize("m,e,k,d,f,n", SIZES)
def test_layer(M, m, e, k, d, f, n, kind, router_kind, act, normalize):
    for pad in (0, 3):
        x, router, w = layer(m, e, d, f, n, kind, router_kind, m + e, pad)
        check(M, x, router, w, k, act, normalize, kind)


def test_result_types_and_every_token_on_one_expert(M):
    x, router, w = layer(40, 6, 256, 96, 64, "bf16", "f32", 3)
    router[:] = 0
    router[4, 0] = 1.0
    x[:, 0] = 30.0
    for kind in ("bf16", "f16", "f32"):
        check(M, x, router, w, 1, "silu", True, kind)
        check(M, x, router, w, 3, "silu", True, kind)  # ties below the first


def test_equal_logits_go_to_the_lowest_index(M):
    x, router, w = layer(20, 130, 64, 48, 32, "f16", "f16", 3)
    router[1:] = router[0]
    y = check(M, x, router, w, 7, "relu", True, "f16")
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("m,e,k,d,f,n", [(4, 64, 32, 64, 48, 20), (4, 65, 32, 64, 48, 20), (5, 64, 32, 64, 48, 20), (2, 64, 64 // 2, 15, 520, 5),
                                         (3, 40, 9, 200, 15, 4100), (1, 33, 1, 100, 511, 3), (4, 7, 7, 33, 513, 9000),
                                         (4, 64, 8, 300, 16, 1)])
def test_few_tokens(M, m, e, k, d, f, n):
    for kind in ("bf16", "f32"):
        x, router, w = layer(m, e, d, f, n, kind, "f32", 17, 1)
        check(M, x, router, w, k, "silu", True, kind)


@pytest.mark.parametrize("m,e,k,d,f,n", [(64, 2, 2, 64, 16384 + 33, 5), (40, 4, 2, 70, 8200, 17), (33, 8, 4, 129, 4096, 16)])
def test_many_channels_and_tokens(M, m, e, k, d, f, n):
    """Enough of both for workgroups of 64 channels, some of them beyond the last."""
    x, router, w = layer(m, e, d, f, n, "f16", "f32", 23, 3)
    check(M, x, router, w, k, "silu", False, "f16")


@pytest.mark.parametrize("m", [3, 9])
def test_choices_of_nearly_equal_logits(M, m):
    """Logits that are equal in 32 bits and differ in 64, in no order of their
    experts, beside exactly equal ones and NaN."""
    e, d = 48, 64
    x, router, w = layer(m, e, d, 32, 24, "f32", "f32", 8)
    x[:, :3] = torch.tensor([1.0, 2.0 ** -20, 2.0 ** -20], device="cuda")
    router.zero_()
    router[:, 0] = 1.0
    g = torch.Generator(device="cuda").manual_seed(1)
    router[:, 1] = (torch.randperm(e, device="cuda", generator=g) // 2) * 2.0 ** -20
    router[5, 2] = router[5, 1]
    check(M, x, router, w, 12, "silu", True, "f32")
    check(M, x, router, w, 12, "silu", False, "f32")
    router[7, 0] = float("nan")  # of every token
    experts, y = torch.empty(m, 12, dtype=torch.int32, device="cuda"), torch.empty(m, 24, device="cuda")
    p = torch.empty(m, 12, device="cuda")
    M.few(x, router, *w, y, 12, experts=experts, weights=p)
    assert torch.equal(experts.long(), R.choose(x, router, 12, True)[0]) and p.isnan().all() and bool((experts[:, 0] == 7).all())


def test_rows_that_are_not_finite(M):
    x, router, w = layer(6, 8, 200, 90, 50, "bf16", "f32", 5)
    good, y = x.clone(), torch.empty(6, 50, device="cuda")
    x[1, 3] = float("nan")
    x[4, 7] = float("inf")
    experts = torch.full((6, 2), -9, dtype=torch.int32, device="cuda")
    M.few(x, router, *w, y, 2, experts=experts)
    assert y[1].isnan().all() and y[4].isnan().all()
    assert bool((experts >= 0).all()) and bool((experts < 8).all())
    _, _, want, bound = R.layer(good, router, *w, 2, "silu", True, "f32")
    for r in (0, 2, 3, 5):
        assert ((y[r].double() - want[r]).abs() <= bound[r]).all()
    x, router, w = layer(3, 8, 64, 32, 16, "f32", "f32", 6)
    x[1] = 0  # a row of zeros: all logits equal, all hidden values 0
    y = torch.empty(3, 16, device="cuda")
    M.few(x, router, *w, y, 2)
    assert not y[1].any() and y[0].any()


def test_codes_beyond_32_bits(M):
    """Experts that lie further apart than 2^32 bytes."""
    e, d, f, n, far = 3, 256, 48, 32, (1 << 31) + 4096 + 7
    x, router, w = layer(9, e, d, f, n, "bf16", "f32", 8)
    room = torch.empty(2 * far + f * d, dtype=torch.int8, device="cuda")
    for i in (0, 2, 4):
        v = w[i]
        spread = room.as_strided(v.shape, (far, v.shape[2], 1))
        spread.copy_(v)
        check(M, x, router, w[:i] + [spread] + w[i + 1:], 2, "silu", True, "bf16")


def test_streams_and_graph(M):
    x, router, w = layer(5, 16, 512, 256, 384, "bf16", "f32", 9)
    y, ex, p = torch.empty(5, 384, device="cuda"), torch.empty(5, 3, dtype=torch.int32, device="cuda"), torch.empty(5, 3, device="cuda")
    results = (y, ex, p)
    run = lambda stream=None: M.few(x, router, *w, y, 3, experts=ex, weights=p, stream=stream)  # noqa: E731
    run()
    want = [t.clone() for t in results]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0):
        for t in results:
            t.zero_()
        torch.cuda.synchronize()
        run(stream)
        torch.cuda.synchronize()
        assert all(torch.equal(a, t) for a, t in zip(results, want))
    # two graphs that share a workspace, replayed in turn
    room = M.workspace_bytes(x, router, *w, 3)
    ws = torch.empty(room, dtype=torch.uint8, device="cuda")
    x2, router2, w2 = layer(4, 16, 512, 200, 100, "bf16", "f32", 10)
    y2 = torch.empty(4, 100, device="cuda")
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        M.few(x, router, *w, y, 3, experts=ex, weights=p, workspace=ws)
    with torch.cuda.graph(graphs[1]):
        M.few(x2, router2, *w2, y2, 2, workspace=ws)
    for s in range(4):
        x.copy_(layer(5, 16, 512, 8, 8, "bf16", "f32", 90 + s)[0])
        x2.copy_(layer(4, 16, 512, 8, 8, "bf16", "f32", 95 + s)[0])
        for t in (*results, y2):
            t.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (*results, y2)]
        run()
        M.few(x2, router2, *w2, y2, 2)
        assert all(torch.equal(a, t) for a, t in zip((*results, y2), got))


def plan_of(E, e, d, f, n, seed=40):
    specs = []
    for i in range(e):
        specs += [synth.random_int8_tensor(r, c, 2.0, seed + 3 * i + j, c * 2) for j, (r, c) in enumerate(((f, d), (f, d), (n, f)))]
    for sp in specs:
        sp["scales"] = (np.asarray(sp["scales"], np.float32) / np.abs(sp["scales"]).max() * 0.02).astype(np.float32)
    b = E.encode_batch(specs, n_threads=4)
    p = E.plan(b.tensors, b.freq, b.chunks, b.blob.size)
    scales = torch.from_numpy(np.concatenate([sp["scales"] for sp in specs])).cuda()
    ws = []
    for j, (r, c) in enumerate(((f, d), (f, d), (n, f))):
        ws += [torch.stack([torch.from_numpy(np.asarray(specs[3 * i + j]["symbols"]).view(np.int8).reshape(r, c)) for i in range(e)]).cuda(),
               torch.stack([torch.from_numpy(specs[3 * i + j]["scales"]) for i in range(e)]).cuda()]
    return b, p, torch.from_numpy(b.blob).cuda(), scales, ws


@pytest.mark.parametrize("m", [1, 7, 64, 150])
def test_layer_on_a_plan(E, M, m):
    from entropy_coded_weight_amd.feed_forward import FeedForward
    e, d, f, n, k = 5, 192, 128, 80, 2
    b, p, blob, scales, w = plan_of(E, e, d, f, n)
    torch.manual_seed(m)
    x, router = torch.randn(m, d, device="cuda").bfloat16(), torch.randn(e, d, device="cuda")
    mix = M.MixtureOfExperts(p, scales, router, k, "gelu")
    status = torch.full((p.n_chunks,), -1, dtype=torch.int32, device="cuda")
    mix.decode(blob, status)
    y, ex, pr = torch.empty(m, n, device="cuda"), torch.empty(m, k, dtype=torch.int32, device="cuda"), torch.empty(m, k, device="cuda")
    mix.forward(x, y, ex, pr)
    assert (status == 0).all()
    want = torch.empty_like(y)
    for r in range(0, m, 64):
        M.few(x[r:r + 64], router, *w, want[r:r + 64], k, "gelu")
    assert torch.equal(y, want)
    # the layer is the weighted sum of its experts' feed-forward blocks
    _, _, ref, bound = R.layer(x, router, *w, k, "gelu", True, "f32")
    total = torch.zeros(m, n, dtype=torch.float64, device="cuda")
    for i in range(e):
        one = one_expert(E, b, i)
        block = FeedForward(one, scales[i * (2 * f + n):(i + 1) * (2 * f + n)], "gelu", hidden_type=torch.float32)
        block.decode(blob)
        o = torch.empty(m, n, device="cuda")
        block.forward(x, o)
        total += torch.where(ex == i, pr, 0).sum(1, keepdim=True).double() * o.double()
    assert ((total - y.double()).abs() <= 2 * bound).all()
    # on a stream and a code buffer of the caller
    side, codes = torch.cuda.Stream(), torch.empty(p.out_elems, dtype=torch.int8, device="cuda")
    other, y2 = M.MixtureOfExperts(p, scales, router, k, "gelu", codes=codes), torch.empty_like(y)
    torch.cuda.synchronize()
    other.decode(blob, stream=side)
    other.forward(x, y2, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(y2, y)


def one_expert(E, b, i):
    """The plan of expert i alone, in the same blob."""
    t = b.tensors[3 * i:3 * i + 3].copy()
    t["out_elem_offset"] -= t["out_elem_offset"][0]
    t["scale_row_offset"] -= t["scale_row_offset"][0]
    c = b.chunks[(b.chunks["tensor"] >= 3 * i) & (b.chunks["tensor"] < 3 * i + 3)].copy()
    c["tensor"] -= 3 * i
    return E.plan(t, np.asarray(b.freq).reshape(-1, 256)[3 * i:3 * i + 3], c, b.blob.size)


def test_plans_that_are_no_mixture(E, M):
    b, p, blob, scales, w = plan_of(E, 2, 64, 32, 48)
    router = torch.zeros(2, 64, device="cuda")
    for k in (dict(top_k=3), dict(top_k=0), dict(activation="tanh"), dict(router=router[:1]), dict(router=router.cpu()),
              dict(router=router.int()), dict(codes=torch.empty(10, dtype=torch.int8, device="cuda"))):
        a = dict(router=router, top_k=1)
        a.update(k)
        with pytest.raises(E.EntqError):
            M.MixtureOfExperts(p, scales, **a)
    with pytest.raises(E.EntqError):
        M.MixtureOfExperts(p, scales[:5], router, 1)
    # gates first: not expert by expert
    order = [0, 3, 1, 4, 2, 5]
    specs = [dict(kind=E.KIND_INT8, rows=r, cols=c, symbols=np.zeros(r * c, np.uint8), chunk_symbols=4096,
                  scales=np.ones(r, np.float32)) for r, c in [[(32, 64), (32, 64), (48, 32)] * 2][0]]
    b2 = E.encode_batch([specs[i] for i in order], n_threads=2)
    p2 = E.plan(b2.tensors, b2.freq, b2.chunks, b2.blob.size)
    with pytest.raises(E.EntqError):
        M.MixtureOfExperts(p2, torch.ones(p2.scale_rows, device="cuda"), router, 1)
    mix = M.MixtureOfExperts(p, scales, router, 1)
    x = torch.zeros(3, 64, device="cuda")
    for bad in (lambda: mix.forward(x[:, :63], x), lambda: mix.forward(x, x), lambda: mix.forward(x, torch.zeros(3, 48, device="cuda"), x),
                lambda: mix.forward(x.clone().requires_grad_(), torch.zeros(3, 48, device="cuda"))):
        with pytest.raises(E.EntqError):
            bad()


def test_refusals(E, M):
    x, router, w = layer(4, 6, 64, 48, 32, "bf16", "f32", 1)
    y = torch.empty(4, 32, device="cuda")
    ok = dict(x=x, router=router, gate=w[0], gate_scales=w[1], up=w[2], up_scales=w[3], down=w[4], down_scales=w[5], y=y, top_k=2)
    bad = [dict(x=torch.zeros(65, 64, device="cuda")), dict(x=x.double()), dict(x=x.float().requires_grad_()), dict(x=x[:, :63]),
           dict(router=router[:5]), dict(router=router.t()), dict(router=router.int()), dict(gate=w[0][0]), dict(gate=w[0].int()),
           dict(gate=w[0].transpose(1, 2)), dict(gate=w[0][:1].expand(6, 48, 64)), dict(gate=w[0].cpu()), dict(up=w[2][:, :47]),
           dict(down=w[4][:, :, :47]), dict(down=w[4][:5]), dict(gate_scales=w[1][:, :47]), dict(gate_scales=w[1].half()),
           dict(up_scales=w[3].t().contiguous().t()), dict(down_scales=w[5][:1].expand(6, 32)), dict(top_k=0), dict(top_k=7),
           dict(top_k=1.5), dict(activation="tanh"), dict(y=y[:3]), dict(y=y.double()), dict(y=y[:, :31]),
           dict(experts=torch.zeros(4, 2, device="cuda")), dict(experts=torch.zeros(4, 3, dtype=torch.int32, device="cuda")),
           dict(weights=torch.zeros(4, 2, device="cuda").half()), dict(weights=torch.zeros(2, 4, device="cuda").t()),
           dict(workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))]
    for i, k in enumerate(bad):
        with pytest.raises(E.EntqError) as e:
            M.few(**{**ok, **k})
        assert e.value.status == E.EINVAL, i
    M.few(**{**ok, "x": x[:0], "y": y[:0]})
