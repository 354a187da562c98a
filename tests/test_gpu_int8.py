"""GPU tests of the int8 products against their formulas in 64 bits
(int8_reference): the quantiser and the product bit for bit, the gated kernel
and the gradients within bounds derived from their roundings."""
import numpy as np
import pytest
import torch

import int8_reference as R

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(scope="module")
def I():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    from entropy_coded_weight_amd import int8
    return int8


def _say(*what):
    print("[gpu-int8]", *what, flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return t.detach().cpu().to(torch.float64).numpy() if t.is_floating_point() else t.cpu().numpy()


def codes(rng, n, k, full=False):
    if full:
        return rng.integers(-128, 128, (n, k)).astype(np.int8)
    return np.clip(np.rint(rng.laplace(0, 3, (n, k))), -127, 127).astype(np.int8)


def scales(rng, n):
    s = (0.02 * np.exp(0.3 * rng.standard_normal(n))).astype(np.float32)
    s[rng.random(n) < 0.1] *= -1
    return s


def strided(a, ld, offset):
    """a's values in a device matrix of row stride ld whose first element is
    `offset` elements into its buffer; the gaps hold a value that would show."""
    t = torch.as_tensor(a).cuda()
    m, n = t.shape
    buf = torch.full((offset + m * ld + 64,), 77, dtype=t.dtype, device="cuda")
    v = buf[offset:offset + m * ld].view(m, ld)[:, :n]
    v.copy_(t)
    return v


# sides at, below and above the sizes of tiles, matrix instructions and vector loads
SHAPES = [(1, 1, 1), (1, 64, 128), (2, 3, 5), (5, 17, 15), (16, 16, 16), (17, 65, 127), (1, 300, 1024),
          (15, 129, 128), (33, 128, 129), (64, 48, 1040), (65, 257, 64), (100, 100, 100), (128, 256, 256),
          (129, 255, 384), (200, 520, 1031), (257, 300, 272), (300, 64, 2048), (3, 2000, 640),
          (530, 130, 160), (48, 1024, 513)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,k", [(1, 1), (3, 7), (2, 8), (5, 255), (4, 256), (7, 1031), (3, 2048), (2, 4100), (9, 8192),
                                 (1, 28672), (2, 40000), (2, 131071), (300, 65)])
def test_quantize_rows(I, m, k, kind):
    rng = np.random.default_rng(m * 1000 + k)
    x = torch.from_numpy((rng.standard_normal((m, k)) * np.exp(rng.standard_normal((m, 1)) * 4)).astype(np.float32))
    x = x.clamp(-60000, 60000).to(TYPES[kind])
    _say("quantize", m, k, kind)
    q = torch.full((m, k + 3), 99, dtype=torch.int8, device="cuda")
    s = torch.empty(m, device="cuda")
    I.quantize_rows(x.cuda(), q[:, :k], s)
    wq, ws = R.quantize(x.float().numpy())
    assert np.array_equal(s.cpu().numpy(), ws)
    assert np.array_equal(q[:, :k].cpu().numpy(), wq)
    assert (q[:, k:] == 99).all()


def test_quantize_special_rows(I):
    x = np.zeros((11, 40), np.float32)
    x[1, 3] = np.nan
    x[2, 0] = np.inf
    x[3, 39] = -np.inf
    x[4, :] = 1e-42                 # subnormal: below the smallest scale
    x[5, :] = -3.4e38
    x[6, 7] = -0.0
    x[7, :20] = 0.5
    x[7, 20] = 1.0                  # 63.5 steps: rounded half to even
    x[8, :] = 2.0 ** -95
    x[9, :] = np.linspace(-1, 1, 40)
    x[10, 0] = 127.0
    x[10, 1:] = np.arange(39) + 0.5
    for kind in ("f32", "bf16"):
        t = torch.from_numpy(x).to(TYPES[kind])
        q = torch.empty(11, 40, dtype=torch.int8, device="cuda")
        s = torch.empty(11, device="cuda")
        I.quantize_rows(t.cuda(), q, s)
        wq, ws = R.quantize(t.float().numpy())
        assert np.array_equal(s.cpu().numpy(), ws, equal_nan=True)
        assert np.array_equal(q.cpu().numpy(), wq)
        bad = [False, True, True, True, False, kind == "bf16"] + [False] * 5  # (-3.4e38 is no bf16 value)
        assert np.isnan(s.cpu().numpy()).tolist() == bad


def _product(q, sx, w, sw):
    """fp32 results of the product, every rounding as stated."""
    acc = R.sums(q, w).numpy().astype(np.float32)
    return (acc * sx[:, None]).astype(np.float32) * sw


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_bit_for_bit(I, m, n, k, out):
    rng = np.random.default_rng(m + 7 * n + 31 * k)
    w, sw = codes(rng, n, k, full=True), scales(rng, n)
    for kind in ("int8", "bf16", "f32"):
        _say("gemm", m, n, k, kind, out)
        if kind == "int8":
            q, sx = codes(rng, m, k, full=True), scales(rng, m)
            x, xs = dev(q), dev(sx)
        else:
            x, xs = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).to(TYPES[kind]), None
            q, sx = R.quantize(x.float().numpy())
            x = x.cuda()
        y = torch.full((m + 1, n), 9.0, dtype=TYPES[out], device="cuda")
        I.gemm(x, xs, dev(w), dev(sw), y[:m])
        want = torch.from_numpy(_product(q, sx, w, sw)).to(TYPES[out])
        assert torch.equal(y[:m].cpu(), want), kind
        assert (y[m] == 9.0).all()


@pytest.mark.parametrize("m", [1, 40, 150])
@pytest.mark.parametrize("k", [64, 131, 400])
@pytest.mark.parametrize("off,gap", [(0, 64), (0, 16), (1, 0), (3, 5), (16, 7), (4, 4)])
def test_gemm_strides_and_alignments(I, m, k, off, gap):
    rng = np.random.default_rng(off * 100 + gap + k)
    n = 90
    q, w = codes(rng, m, k, True), codes(rng, n, k, True)
    sx, sw = scales(rng, m), scales(rng, n)
    want = torch.from_numpy(_product(q, sx, w, sw))
    _say("strides", m, k, off, gap)
    for xo, wo in ((off, 0), (0, off), (off, off)):
        y = torch.full((m, n + 1 + gap), 5.0, device="cuda")
        I.gemm(strided(q, k + (gap if xo == off else 0), xo), dev(sx), strided(w, k + (gap if wo == off else 0), wo),
               dev(sw), y[:, 1:n + 1])
        assert torch.equal(y[:, 1:n + 1].cpu(), want)
        assert (y[:, 0] == 5).all() and (y[:, n + 1:] == 5).all()


@pytest.mark.parametrize("m", [1, 20, 130])
def test_gemm_largest_sums(I, m):
    """The longest rows: every product at its largest, the int32 sum just
    inside its range."""
    k, n = I.MAX_COLS, 33
    q, w = np.full((m, k), -128, np.int8), np.full((n, k), -128, np.int8)
    w[1] = 127
    one = np.ones
    _say("largest sums", m)
    y = torch.empty(m, n, device="cuda")
    I.gemm(dev(q), dev(one(m, np.float32)), dev(w), dev(one(n, np.float32)), y)
    want = np.full((m, n), np.float32(k * 128 * 128))
    want[:, 1] = np.float32(-k * 128 * 127)
    assert np.array_equal(y.cpu().numpy(), want)


def test_gemm_long_row_stride(I):
    """Rows so far apart that offsets pass 32 bits."""
    rng = np.random.default_rng(3)
    for m in (4, 70):
        n, k, ld = 5, 160, (1 << 30) + 16
        w = codes(rng, n, k, True)
        buf = torch.zeros(4 * ld + k, dtype=torch.int8, device="cuda")
        for i in range(n):
            buf[i * ld:i * ld + k] = dev(w[i])
        far = torch.as_strided(buf, (n, k), (ld, 1))
        q, sx, sw = codes(rng, m, k, True), scales(rng, m), scales(rng, n)
        _say("long stride", m)
        y = torch.empty(m, n, device="cuda")
        I.gemm(dev(q), dev(sx), far, dev(sw), y)
        assert np.array_equal(y.cpu().numpy(), _product(q, sx, w, sw))


def test_empty_sizes(I):
    new = lambda *s, d=torch.float32: torch.full(s, 7.0, device="cuda").to(d)  # noqa: E731
    for m, n, k in ((0, 4, 16), (4, 0, 16), (4, 5, 0), (0, 0, 0)):
        _say("empty", m, n, k)
        x, w = new(m, k, d=torch.int8), new(n, k, d=torch.int8)
        xs, ws = new(m), new(n)
        y = new(m, n)
        I.gemm(x, xs, w, ws, y)
        I.gated(x, xs, w, ws, w, ws, y)
        I.gemm(new(m, k, d=torch.bfloat16), None, w, ws, y)
        assert (y == 0).all() if k == 0 else y.numel() == 0
        I.quantize_rows(new(m, k), x, xs)
        dy, dx = new(m, n, d=torch.bfloat16), new(m, k, d=torch.bfloat16)
        a, b = new(n), new(n)
        I.gemm_backward(dy, x, xs, w, ws, dx, a)
        assert (dx == 0).all() and (a == 0).all()
        dx, a = new(m, k, d=torch.bfloat16), new(n)
        I.gated_backward(dy, x, xs, w, ws, w, ws, dx, a, b)
        assert (dx == 0).all() and (a == 0).all() and (b == 0).all()


def test_many_channels_of_no_columns(I):
    """K = 0 with so many fp32 channels that a row has 2^32 bytes and more:
    every result is 0."""
    n = (1 << 30) + 5
    w, sw = torch.empty(n, 0, dtype=torch.int8, device="cuda"), torch.empty(n, device="cuda")
    x, sx = torch.empty(1, 0, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    y = torch.full((1, n), 3.0, device="cuda")
    I.gemm(x, sx, w, sw, y)
    assert float(y.abs().max()) == 0.0


def _near(got, want, bound, what):
    got = got.detach().to(want.device).double()
    off = (got - want).abs() - bound
    worst = int(off.argmax())
    assert float(off.max()) <= 0, (what, worst, *(float(t.flatten()[worst]) for t in (got, want, bound)))


ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gated(I, m, n, k):
    rng = np.random.default_rng(m + 7 * n + 31 * k)
    q, sx = codes(rng, m, k), scales(rng, m)
    wg, sg, wu, su = codes(rng, n, k), scales(rng, n), codes(rng, n, k), scales(rng, n)
    for i, (name, out) in enumerate(zip(ACTS, ("f32", "bf16", "f16", "f32"))):
        _say("gated", m, n, k, name, out)
        size = np.float32(1 / np.sqrt(k)) * 8  # g around 1, some tails
        h = torch.full((m + 1, n), 9.0, dtype=TYPES[out], device="cuda")
        I.gated(dev(q), dev(sx * size), dev(wg), dev(sg * 20), dev(wu), dev(su), h[:m], name)
        want, err = R.gated(q, sx * size, wg, sg * 20, wu, su, name)
        _near(h[:m], want, err + R.ROUND[out] * want.abs() + R.TINY[out], name)
        assert (h[m] == 9.0).all()


def test_gated_far_activations(I):
    """Gates far out on both sides: results are finite and right."""
    q = np.array([[1], [-1], [100], [-100], [0]], np.int8)
    w = np.array([[127], [1], [-128], [0]], np.int8)
    one5, s = np.ones(5, np.float32), np.array([1.0, 80.0, 0.3, 1e30], np.float32)
    for name in ACTS:
        h = torch.empty(5, 4, device="cuda")
        I.gated(dev(q), dev(one5), dev(w), dev(s), dev(w), dev(np.ones(4, np.float32)), h, name)
        want, err = R.gated(q, one5, w, s, w, np.ones(4), name)
        assert np.isfinite(host(h)).all()
        _near(h, want, err + R.EPS * want.abs() + 1e-37, name)


@pytest.mark.parametrize("m", [1, 40, 200])
def test_gelu_relative_to_itself(I, m):
    """gelu and its derivative keep their relative accuracy where the gate is
    far below 0. g is exact here (a product of 1 and a scale). fp32 roundings:
    exp's argument three (1.5 g^2 EPS), exp and the reciprocal 1 ulp, the
    polynomial 17 EPS with what the reciprocal's error makes of it, three
    products: (24 + 1.5 g^2) EPS of the tail Q(|g|)."""
    rng = np.random.default_rng(m)
    v = np.concatenate([np.linspace(-12, 6, 4001), rng.uniform(-6, 1, 3000), [-1e-30, 0.0, 1e-30]]).astype(np.float32)
    n = len(v)
    one = np.ones((n, 1), np.int8)
    q, sx, ones = np.ones((m, 1), np.int8), np.ones(m, np.float32), np.ones(n, np.float32)
    h = torch.empty(m, n, device="cuda")
    I.gated(dev(q), dev(sx), dev(one), dev(v), dev(one), dev(ones), h, "gelu")
    g = R.f64(v)
    tail = 0.5 * torch.erfc(g.abs() / np.sqrt(2))
    rel = (24 + 1.5 * g * g) * R.EPS * tail
    want = R.act("gelu", v)[0]
    _near(h.cpu(), want.expand(m, n), (g.abs() * rel + 3 * R.EPS * want.abs()).expand(m, n), "gelu")
    # dh = 1, u = 1: the gate scale's gradient is the sum over m of act'(g)
    ds = torch.empty(n, device="cuda")
    I.gated_backward(torch.ones(m, n, device="cuda").half(), dev(q), dev(sx), dev(one), dev(v), dev(one), dev(ones),
                     None, ds, None, "gelu")
    phi = g.abs() * torch.exp(-g * g / 2) / np.sqrt(2 * np.pi)
    want = R.act("gelu", v)[1]
    bound = rel + phi * (6 + 1.5 * g * g) * R.EPS + (m + 8) * R.EPS * want.abs()
    _near(ds.cpu(), m * want, m * bound, "gelu'")


@pytest.mark.parametrize("m,n,k", [(3, 40, 64), (70, 130, 200), (20, 64, 128)])
def test_rows_with_nan_or_infinity_stay_alone(I, m, n, k):
    rng = np.random.default_rng(m)
    x = rng.standard_normal((m, k)).astype(np.float32)
    x[1, 2], x[2, k - 1] = np.nan, -np.inf
    w, sw = codes(rng, n, k), scales(rng, n)
    y, h = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    I.gemm(dev(x), None, dev(w), dev(sw), y)
    I.gated(dev(x), None, dev(w), dev(sw), dev(w), dev(sw), h, "relu")
    bad = np.zeros(m, bool)
    bad[1:3] = True
    for t in (y, h):
        assert np.array_equal(np.isnan(t.cpu().numpy()).any(axis=1), bad)
        assert np.array_equal(np.isnan(t.cpu().numpy()).all(axis=1), bad)
    # a NaN in one token's gradient reaches that token's dX and no other's
    q, sx = R.quantize(rng.standard_normal((m, k)))
    for kind in ("bf16", "f16"):
        dy = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).to(TYPES[kind]).cuda()
        dy[1, n - 1] = float("nan")
        dx = torch.empty(m, k, dtype=TYPES[kind], device="cuda")
        I.gated_backward(dy, dev(q), dev(sx), dev(w), dev(sw), dev(w), dev(sw), dx)
        nan = np.isnan(host(dx))
        assert not nan[0].any() and not nan[2:].any() and nan[1].any()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("n,k", [(33, 1), (40, 127), (70, 1031), (50, 8192), (41, 8225), (20, 32768), (20, 32769),
                                 (16384, 96), (16385, 96)])
def test_one_token_of_activations(I, n, k, kind):
    """One token that the call quantises itself, in the product's kernel or
    before it: the plain product bit for bit, the gated one within its bound."""
    rng = np.random.default_rng(n + k)
    wg, sg, wu, su = codes(rng, n, k), scales(rng, n), codes(rng, n, k), scales(rng, n)
    _say("one token", n, k, kind)
    for off in (0, 1):
        x = torch.from_numpy(rng.standard_normal((1, k)).astype(np.float32)).to(TYPES[kind])
        q, sx = R.quantize(x.float().numpy())
        size = np.float32(50 / np.sqrt(k))
        xd = strided(x, k + off, off)
        w, w2 = strided(wg, k + off, off), strided(wu, k + 2 * off, 3 * off)
        y = torch.full((2, n), 9.0, device="cuda")
        I.gemm(xd, None, w, dev(sg), y[:1])
        assert np.array_equal(y[:1].cpu().numpy(), _product(q, sx, wg, sg))
        for i, name in enumerate(ACTS):
            out = ("f32", "bf16", "f16", "f32")[i]
            h = torch.full((2, n), 9.0, dtype=TYPES[out], device="cuda")
            I.gated(xd, None, w, dev(sg * size), w2, dev(su), h[:1], name)
            want, err = R.gated(q, sx, wg, sg * size, wu, su, name)
            _near(h[:1].cpu(), want, err + R.ROUND[out] * want.abs() + R.TINY[out], name)
            assert (h[1] == 9.0).all()
        assert (y[1] == 9.0).all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
def test_one_bad_token(I, kind, bad):
    rng = np.random.default_rng(1)
    n, k = 90, 1500
    x = torch.from_numpy(rng.standard_normal((1, k)).astype(np.float32)).to(TYPES[kind])
    x[0, 777] = float(bad)
    w, sw = dev(codes(rng, n, k)), dev(scales(rng, n))
    y, h = torch.empty(1, n, device="cuda"), torch.empty(1, n, device="cuda")
    I.gemm(x.cuda(), None, w, sw, y)
    I.gated(x.cuda(), None, w, sw, w, sw, h, "gelu")
    assert torch.isnan(y).all() and torch.isnan(h).all()


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_gemm_of_f16_activations_bit_for_bit(I, m, n, k):
    rng = np.random.default_rng(m + 7 * n + 31 * k)
    w, sw = codes(rng, n, k, full=True), scales(rng, n)
    x = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).half()
    q, sx = R.quantize(x.float().numpy())
    y = torch.empty(m, n, device="cuda")
    I.gemm(x.cuda(), None, dev(w), dev(sw), y)
    assert np.array_equal(y.cpu().numpy(), _product(q, sx, w, sw))


@pytest.mark.parametrize("m", [2, 40, 130])
def test_gated_of_activations(I, m):
    """Several tokens of activations against their codes, every type."""
    rng = np.random.default_rng(m)
    n, k = 150, 333
    wg, sg, wu, su = codes(rng, n, k), scales(rng, n), codes(rng, n, k), scales(rng, n)
    for kind in TYPES:
        x = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).to(TYPES[kind])
        q, sx = R.quantize(x.float().numpy())
        for name in ACTS:
            h = torch.empty(m, n, device="cuda")
            I.gated(x.cuda(), None, dev(wg), dev(sg), dev(wu), dev(su), h, name)
            want, err = R.gated(q, sx, wg, sg, wu, su, name)
            _near(h.cpu(), want, err + R.EPS * want.abs() + R.TINY["f32"], (kind, name))


BACK = [(1, 1, 1), (2, 70, 16), (17, 64, 65), (64, 130, 128), (65, 63, 200), (130, 257, 96), (257, 128, 272),
        (40, 300, 1031), (300, 520, 256), (1, 1000, 512), (600, 33, 33), (16, 1024, 48)]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", BACK)
def test_gemm_backward(I, m, n, k, kind):
    rng = np.random.default_rng(m + 5 * n + 11 * k)
    q, sx, w, sw = codes(rng, m, k), scales(rng, m), codes(rng, n, k, True), scales(rng, n)
    dy = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).to(TYPES[kind])
    _say("gemm_backward", m, n, k, kind)
    dx = torch.full((m + 1, k), 9.0, dtype=TYPES[kind], device="cuda")
    ds = torch.empty(n, device="cuda")
    I.gemm_backward(dy.cuda(), dev(q), dev(sx), dev(w), dev(sw), dx[:m], ds)
    (wx, bx), (ws, bs) = R.gemm_backward(host(dy), q, sx, w, sw, kind)
    _near(dx[:m], wx, bx, "dx")
    _near(ds, ws, bs, "dsw")
    assert (dx[m] == 9.0).all()
    # each gradient alone is the same
    dx2, ds2 = torch.empty_like(dx[:m]), torch.empty_like(ds)
    I.gemm_backward(dy.cuda(), dev(q), dev(sx), dev(w), dev(sw), dx2)
    I.gemm_backward(dy.cuda(), dev(q), dev(sx), dev(w), dev(sw), None, ds2)
    assert torch.equal(dx2, dx[:m]) and torch.equal(ds2, ds)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", BACK)
def test_gated_backward(I, m, n, k, kind):
    rng = np.random.default_rng(m + 5 * n + 11 * k)
    size = np.float32(20 / np.sqrt(k))
    q, sx = codes(rng, m, k), scales(rng, m) * size
    wg, sg, wu, su = codes(rng, n, k), scales(rng, n) * 8, codes(rng, n, k), scales(rng, n)
    dh = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).to(TYPES[kind])
    for name in ACTS:
        _say("gated_backward", m, n, k, kind, name)
        dx = torch.full((m + 1, k), 9.0, dtype=TYPES[kind], device="cuda")
        dsg, dsu = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
        args = (dh.cuda(), dev(q), dev(sx), dev(wg), dev(sg), dev(wu), dev(su))
        I.gated_backward(*args, dx[:m], dsg, dsu, name)
        ends = R.gated_backward(host(dh), q, sx, wg, sg, wu, su, name, kind)
        for got, (want, bound), what in zip((dx[:m], dsg, dsu), ends, ("dx", "dsg", "dsu")):
            _near(got, want, bound, (name, what))
        assert (dx[m] == 9.0).all()
        dx2, g2, u2 = torch.empty_like(dx[:m]), torch.empty_like(dsg), torch.empty_like(dsu)
        I.gated_backward(*args, dx2, activation=name)
        I.gated_backward(*args, None, g2, None, name)
        I.gated_backward(*args, None, None, u2, name)
        assert torch.equal(dx2, dx[:m]) and torch.equal(g2, dsg) and torch.equal(u2, dsu)


@pytest.mark.parametrize("m", [3, 70, 600])
@pytest.mark.parametrize("name", ACTS)
def test_far_gates_backward(I, m, name):
    """Gates so far out that act' is 0 or 1 to the last bit and g^2 is beyond
    fp32 (or exactly 0): the gradients are finite and right."""
    rng = np.random.default_rng(m)
    n, k = 130, 64
    q, wg, wu = codes(rng, m, k), codes(rng, n, k), codes(rng, n, k)
    sx, sg, su = np.full(m, 0.01, np.float32), np.full(n, 1e25, np.float32), np.abs(scales(rng, n)) * np.float32(1e-20)
    sg[::3] = 1e21
    g0, u0 = R.sums(q, wg) * R.f64(sx)[:, None], R.sums(q, wu) * R.f64(sx)[:, None]
    g, u = g0 * R.f64(sg), u0 * R.f64(su)
    dh = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).bfloat16()
    dx = torch.empty(m, k, dtype=torch.bfloat16, device="cuda")
    a, b = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    I.gated_backward(dh.cuda(), dev(q), dev(sx), dev(wg), dev(sg), dev(wu), dev(su), dx, a, b, name)
    act, grad = R.act(name, g)
    dg, du = R.f64(dh) * u * grad, R.f64(dh) * act
    want, bound = R._dx([dg, du], [0 * dg, 0 * du], [R.f64(sg), R.f64(su)], [wg, wu], "bf16")
    _near(dx.cpu(), want, bound + R.EPS * 20 * want.abs(), "dx")
    for got, d, raw in ((a, dg, g0), (b, du, u0)):
        t = d * raw
        _near(got.cpu(), t.sum(0), (m + 30) * R.EPS * t.abs().sum(0) + 1e-44, "ds")


@pytest.mark.parametrize("off,gap", [(1, 0), (2, 3), (16, 16)])
@pytest.mark.parametrize("m,k", [(3, 64), (150, 201)])
def test_backward_strides(I, m, k, off, gap):
    rng = np.random.default_rng(off + gap + m)
    n = 77
    q, sx, w, sw = codes(rng, m, k), scales(rng, m), codes(rng, n, k), scales(rng, n)
    dy = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).to(torch.bfloat16)
    dx = torch.full((m, k + 2 + gap), 5.0, dtype=torch.bfloat16, device="cuda")
    ds = torch.empty(n, device="cuda")
    _say("backward strides", m, k, off, gap)
    I.gemm_backward(strided(dy, n + gap, off), strided(q, k + gap, off), dev(sx), strided(w, k + gap, off), dev(sw),
                    dx[:, 1:k + 1], ds)
    (wx, bx), (ws, bs) = R.gemm_backward(host(dy), q, sx, w, sw, "bf16")
    _near(dx[:, 1:k + 1], wx, bx, "dx")
    _near(ds, ws, bs, "dsw")
    assert (dx[:, 0] == 5).all() and (dx[:, k + 1:] == 5).all()


@pytest.mark.parametrize("top", [1e-5, 1e9])
def test_f16_gradients_do_not_leave_their_range(I, top):
    """Channel scales far below or above 1 neither flush dy sw to zero nor
    overflow it: dX is scaled by a power of two while it is in 16 bits."""
    rng = np.random.default_rng(8)
    m, n, k = 20, 96, 64
    q, sx, w = codes(rng, m, k), scales(rng, m), codes(rng, n, k)
    sw = (scales(rng, n) * np.float32(top)).astype(np.float32)
    dy = torch.from_numpy((rng.standard_normal((m, n)) * min(1e3, 1e-3 / top)).astype(np.float32)).half()
    if top > 1:
        dy = torch.zeros_like(dy)
        dy[:, :3] = 6e-8  # the smallest f16 value
    dx = torch.empty(m, k, dtype=torch.float16, device="cuda")
    I.gemm_backward(dy.cuda(), dev(q), dev(sx), dev(w), dev(sw), dx)
    wx, bx = R.gemm_backward(host(dy), q, sx, w, sw, "f16")[0]
    fits = wx.abs() < 60000
    got = dx.cpu().double()
    assert bool(((got - wx).abs()[fits] <= bx[fits]).all())


# tokens and sides that take the few-token kernel, whole and split tiles, and
# every way in which scaled gradients get into 16 bits
RANGE = [(1, 1, 1), (3, 70, 33), (40, 300, 1031), (96, 1000, 4112), (300, 520, 256), (1100, 2100, 300)]


def _f16_ends(d, scales_of, weights):
    """dX = sum over t of (d_t s_t) w_t for F16, with a bound that knows no more
    of a row than the row itself: each d s rounded to 11 bits, or to steps of
    2^-24 once the token's largest is in [2^14, 2^15), fp32 sums in any order."""
    n = weights[0].shape[0]
    ds = [v * R.f64(s) for v, s in zip(d, scales_of)]
    top = torch.stack([v.abs().amax(1) for v in ds]).amax(0)
    dx, bound = 0.0, 0.0
    for v, w in zip(ds, weights):
        w = R.f64(w)
        dx = dx + v @ w
        bound = bound + (v.abs() * (R.ROUND["f16"] + (2 * n + 30) * R.EPS) + 2.0 ** -39 * top[:, None]) @ w.abs()
    return dx, bound + R.ROUND["f16"] * dx.abs() + R.TINY["f16"]


def _f16_product(I, dy, q, sx, w, sw):
    m, n, k = *dy.shape, q.shape[1]
    dx, alone = (torch.empty(m, k, dtype=torch.float16, device="cuda") for _ in range(2))
    ds = torch.empty(n, device="cuda")
    args = (dy.cuda(), dev(q), dev(sx), dev(w), dev(sw))
    I.gemm_backward(*args, dx, ds)
    I.gemm_backward(*args, alone)
    assert torch.equal(dx, alone)
    want, bound = _f16_ends([R.f64(dy)], [sw], [w])
    assert float(want.abs().max()) < 65000
    _near(dx.cpu(), want, bound, "dx")


@pytest.mark.parametrize("m,n,k", RANGE)
def test_f16_product_gradients_of_any_size(I, m, n, k):
    """dY up to F16's largest value, tokens of very different size, and a
    channel whose scale stands far out but which adds nothing to dX."""
    rng = np.random.default_rng(m + n + k)
    q, sx, w = codes(rng, m, k), scales(rng, m), codes(rng, n, k)
    sw = (np.float32(0.0155 / 8 / np.sqrt(n)) * rng.uniform(0.5, 1, n)).astype(np.float32)
    _say("f16 product, large", m, n, k)
    dy = torch.from_numpy(rng.choice([-1.0, 1.0], (m, n)) * rng.uniform(40000, 65504, (m, n))).half()
    _f16_product(I, dy, q, sx, w, sw)
    _say("f16 product, tokens apart", m, n, k)
    dy = dy / torch.from_numpy(2.0 ** rng.integers(0, 28, (m, 1))).float()
    _f16_product(I, dy.half(), q, sx, w, sw)
    for far in (1e4, 1e8):
        _say("f16 product, one scale far out", m, n, k, far)
        dy = torch.from_numpy(rng.standard_normal((m, n)) * 1e-3).half()
        sw = (0.01 * rng.uniform(0.5, 1, n)).astype(np.float32)
        sw[n // 2] = far * 0.01
        dy[:, n // 2] = 0
        _f16_product(I, dy, q, sx, w, sw)
        dy[:, n // 2] = 1e-3
        w[n // 2] = 0
        if far == 1e4:  # (the row's largest is this channel's: others keep 11 bits to 2^-29 of it)
            _f16_product(I, dy, q, sx, w, sw)


def _f16_gated(I, dh, q, sx, wg, sg, wu, su):
    """relu, whose values and gradients carry no error of their own."""
    m, n, k = *dh.shape, q.shape[1]
    dx, alone = (torch.empty(m, k, dtype=torch.float16, device="cuda") for _ in range(2))
    a, b = torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    args = (dh.cuda(), dev(q), dev(sx), dev(wg), dev(sg), dev(wu), dev(su))
    I.gated_backward(*args, dx, a, b, "relu")
    I.gated_backward(*args, alone, activation="relu")
    assert torch.equal(dx, alone)
    g0, u0 = R.sums(q, wg) * R.f64(sx)[:, None], R.sums(q, wu) * R.f64(sx)[:, None]
    h, dh = R.f64(dh), (g0 * R.f64(sg) > 0)
    dg, du = h * dh * u0 * R.f64(su), h * dh * g0 * R.f64(sg)
    want, bound = _f16_ends([dg, du], [sg, su], [wg, wu])
    assert float(want.abs().max()) < 65000
    _near(dx.cpu(), want, bound, "dx")
    for got, d, raw in ((a, dg, g0), (b, du, u0)):
        t = d * raw
        _near(got.cpu(), t.sum(0), (m + 30) * R.EPS * t.abs().sum(0) + 1e-44, "ds")


@pytest.mark.parametrize("m,n,k", RANGE)
def test_f16_gated_gradients_of_any_size(I, m, n, k):
    """Gates and up values far beyond F16's range of dh times them, tokens of
    very different size, gate and up scales of very different size, and a
    channel far out that adds nothing to dX."""
    rng = np.random.default_rng(2 * m + n + k)
    q, wg, wu = codes(rng, m, k), codes(rng, n, k), codes(rng, n, k)
    near = lambda size: (size * rng.uniform(0.5, 1, n)).astype(np.float32)  # noqa: E731
    sx = near(1)[:1].repeat(m) * np.float32(8 / (3 * 4 * 3 * 4 * np.sqrt(k)))  # sums times sx around 1
    dh = torch.from_numpy(64 * rng.standard_normal((m, n))).half()
    _say("f16 gated, large", m, n, k)
    # g and u of some 2000, dg and du of some 10^5
    small = 1e-3 / np.sqrt(n)
    _f16_gated(I, dh, q, sx * np.float32(2000 / small), wg, near(small), wu, near(small))
    _say("f16 gated, tokens apart", m, n, k)
    rows = (2.0 ** -rng.integers(0, 20, m)).astype(np.float32)
    _f16_gated(I, dh, q, sx * np.float32(2000 / small) * rows, wg, near(small), wu, near(small))
    _say("f16 gated, up far below gate", m, n, k)
    _f16_gated(I, dh / 6.4e6, q, sx, wg, near(1e3), wu, near(1e-3))
    _f16_gated(I, dh / 6.4e6, q, sx, wg, near(1e-3), wu, near(1e3))
    _say("f16 gated, one scale far out", m, n, k)
    sg, su = near(1e-2), near(1e-2)
    sg[n // 2] = su[n - 1] = 1e6
    dh[:, n // 2] = dh[:, n - 1] = 0
    _f16_gated(I, dh / 64, q, sx, wg, sg, wu, su)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m", [3, 40, 300])
def test_an_infinite_gradient_gives_infinities(I, m, kind):
    """One infinity in dY: dX of that token is an infinity of the code's sign,
    NaN where the code is 0, and no other token sees it."""
    rng = np.random.default_rng(m)
    n, k = 200, 96
    q, sx, w, sw = codes(rng, m, k), scales(rng, m), codes(rng, n, k), np.abs(scales(rng, n))
    dy = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).to(TYPES[kind])
    dy[1, 7] = float("inf")
    dx = torch.empty(m, k, dtype=TYPES[kind], device="cuda")
    I.gemm_backward(dy.cuda(), dev(q), dev(sx), dev(w), dev(sw), dx, torch.empty(n, device="cuda"))
    want = np.where(w[7] > 0, np.inf, np.where(w[7] < 0, -np.inf, np.nan))
    assert np.array_equal(host(dx)[1], want, equal_nan=True)
    assert np.isfinite(np.delete(host(dx), 1, axis=0)).all()


# products that take every tile size, whole and with the sum split, each with
# sides that end inside a tile; 64-bit references on the GPU
LARGE = [(1100, 8200, 272), (520, 2001, 4096), (700, 16390, 1040), (256, 8192, 28672), (1000, 5000, 4000),
         (512, 8190, 28672), (25, 2000, 2048), (40, 3000, 640), (3001, 300, 2064)]


def _large(m, n, k, seed, weights):
    g = torch.Generator(device="cuda").manual_seed(seed)
    code = lambda *s: torch.randint(-128, 128, s, generator=g, device="cuda", dtype=torch.int8)  # noqa: E731
    scale = lambda r: (torch.rand(r, generator=g, device="cuda") + 0.5) * 0.01  # noqa: E731
    q = code(m, k)
    sx = scale(m) * (4.0 / (k ** 0.5 * 74 * 74 * 0.01 * 0.01))  # |g| up to 10 or so
    return (q, sx) + tuple(t for _ in range(weights) for t in (code(n, k), scale(n)))


@pytest.mark.parametrize("m,n,k", LARGE)
def test_large_forward(I, m, n, k):
    _say("large forward", m, n, k)
    q, sx, wg, sg, wu, su = _large(m, n, k, m + n, 2)
    y = torch.full((m + 1, n + 3), 7.0, device="cuda")
    I.gemm(q, sx, wg, sg, y[:m, :n])
    acc = R.sums(q, wg).float()
    assert torch.equal(y[:m, :n], acc * sx[:, None] * sg)
    assert (y[m] == 7).all() and (y[:, n:] == 7).all()
    for out in ("f32", "bf16"):
        h = torch.full((m + 1, n + 3), 7.0, device="cuda").to(TYPES[out])
        I.gated(q, sx, wg, sg, wu, su, h[:m, :n], "gelu")
        want, err = R.gated(q, sx, wg, sg, wu, su, "gelu")
        _near(h[:m, :n], want, err + R.ROUND[out] * want.abs() + R.TINY[out], out)
        assert (h[m] == 7).all() and (h[:, n:] == 7).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m,n,k", [(1100, 8200, 272), (520, 2001, 4096), (1000, 5000, 4000), (2050, 3001, 4103),
                                   (256, 8192, 8192), (40, 3000, 640), (90, 200, 4112), (96, 1000, 8192),
                                   (70, 130, 3000)])
def test_large_backward(I, m, n, k, kind):
    _say("large backward", m, n, k, kind)
    q, sx, wg, sg, wu, su = _large(m, n, k, m + n, 2)
    dh = (torch.randn(m, n, device="cuda") * 0.1).to(TYPES[kind])
    new = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    dx, ds = new(m + 1, k + 3).to(TYPES[kind]), new(n)
    I.gemm_backward(dh, q, sx, wg, sg, dx[:m, :k], ds)
    for got, (want, bound), what in zip((dx[:m, :k], ds), R.gemm_backward(dh, q, sx, wg, sg, kind), ("dx", "ds")):
        _near(got, want, bound, what)
    dx, dsg, dsu = new(m + 1, k + 3).to(TYPES[kind]), new(n), new(n)
    I.gated_backward(dh, q, sx, wg, sg, wu, su, dx[:m, :k], dsg, dsu, "silu")
    for got, (want, bound), what in zip((dx[:m, :k], dsg, dsu),
                                        R.gated_backward(dh, q, sx, wg, sg, wu, su, "silu", kind), ("dx", "dsg", "dsu")):
        _near(got, want, bound, what)
    assert (dx[m] == 7).all() and (dx[:, k:] == 7).all()


@pytest.mark.parametrize("m,n,k", [(3, 40000, 64), (3, 20000, 64), (100, 5121, 4112), (70000, 5, 16)])
def test_f16_rows_of_every_length(I, m, n, k):
    """Rows longer than what a workgroup keeps of them in registers, beside
    split tiles too, and more tokens than a launch has workgroups for."""
    _say("f16 rows", m, n, k)
    q, sx, wg, sg, wu, su = _large(m, n, k, m + n, 2)
    g = torch.Generator(device="cuda").manual_seed(n)
    dh = (torch.randn(m, n, device="cuda", generator=g) * 0.1).half()
    new = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    dx, ds = new(m + 1, k + 3).half(), new(n)
    I.gemm_backward(dh, q, sx, wg, sg, dx[:m, :k], ds)
    for got, (want, bound), what in zip((dx[:m, :k], ds), R.gemm_backward(dh, q, sx, wg, sg, "f16"), ("dx", "ds")):
        _near(got, want, bound, what)
    dx, dsg, dsu = new(m + 1, k + 3).half(), new(n), new(n)
    I.gated_backward(dh, q, sx, wg, sg, wu, su, dx[:m, :k], dsg, dsu, "silu")
    for got, (want, bound), what in zip((dx[:m, :k], dsg, dsu),
                                        R.gated_backward(dh, q, sx, wg, sg, wu, su, "silu", "f16"), ("dx", "dsg", "dsu")):
        _near(got, want, bound, what)
    assert (dx[m] == 7).all() and (dx[:, k:] == 7).all()


def test_other_stream_given_workspace_and_repeats(I):
    """A stream of the caller, a workspace of the caller with other work's
    leftovers in it, and the same bits on every call."""
    rng = np.random.default_rng(12)
    m, n, k = 70, 200, 300
    x = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).bfloat16().cuda()
    w, sw, w2, sw2 = dev(codes(rng, n, k)), dev(scales(rng, n)), dev(codes(rng, n, k)), dev(scales(rng, n))
    dh = torch.randn(m, n, device="cuda").bfloat16()
    q, sx = torch.empty(m, k, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    I.quantize_rows(x, q, sx)

    def all_of(stream, fill):
        ws = None
        outs = []
        for op, args in (("gated", (x, None, w, sw, w2, sw2)), ("gated_backward", (q, sx, w, sw, w2, sw2))):
            back = op == "gated_backward"
            need = I.workspace_bytes(op, *args, dy=dh if back else None)
            if fill is not None:
                raw = torch.full((need + 256,), fill, dtype=torch.uint8, device="cuda")
                at = -raw.data_ptr() % 256
                ws = raw[at:at + need]
            torch.cuda.synchronize()
            if back:
                o = [torch.full((m, k), 3.0, device="cuda").bfloat16(), torch.zeros(n, device="cuda"),
                     torch.zeros(n, device="cuda")]
                torch.cuda.synchronize()
                I.gated_backward(dh, *args, *o, stream=stream, workspace=ws)
            else:
                o = [torch.empty(m, n, device="cuda")]
                I.gated(*args, o[0], stream=stream, workspace=ws)
            torch.cuda.synchronize()
            outs += o
        return outs

    want = all_of(None, None)
    side = torch.cuda.Stream()
    for stream, fill in ((None, 0xFF), (side, None), (side, 0x7F), (side.cuda_stream, None), (0, 0xFF)):
        for a, b in zip(all_of(stream, fill), want):
            assert torch.equal(a, b)


def test_graph_capture(I):
    """The calls inside a captured graph, replayed between eager calls with
    new inputs."""
    rng = np.random.default_rng(13)
    m, n, k = 24, 320, 256
    x = torch.zeros(m, k, dtype=torch.bfloat16, device="cuda")
    w, sw, w2, sw2 = dev(codes(rng, n, k)), dev(scales(rng, n)), dev(codes(rng, n, k)), dev(scales(rng, n))
    q, sx = torch.empty(m, k, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    h, dx = torch.empty(m, n, dtype=torch.float16, device="cuda"), torch.empty(m, k, dtype=torch.float16, device="cuda")
    ds = [torch.empty(n, device="cuda") for _ in range(2)]

    def step(q, sx, h, dx, ds):
        I.quantize_rows(x, q, sx)
        I.gated(q, sx, w, sw, w2, sw2, h)
        I.gated_backward(h, q, sx, w, sw, w2, sw2, dx, *ds)

    step(q, sx, h, dx, ds)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(q, sx, h, dx, ds)
    for i in range(4):
        x.copy_(torch.randn(m, k, device="cuda"))
        g.replay()
        e = (torch.empty_like(q), torch.empty_like(sx), torch.empty_like(h), torch.empty_like(dx),
             [torch.empty_like(t) for t in ds])
        step(*e)
        torch.cuda.synchronize()
        for a, b in zip((q, sx, h, dx, *ds), (*e[:4], *e[4])):
            assert torch.equal(a, b), i


def test_refusals(I):
    """What the binding refuses on the GPU, before any launch."""
    from entropy_coded_weight_amd import EINVAL, EntqError
    new = lambda *s, d=torch.float32: torch.zeros(s, device="cuda").to(d)  # noqa: E731
    i8, bf = torch.int8, torch.bfloat16
    x, q, sx, w, sw, y = new(4, 32, d=bf), new(4, 32, d=i8), new(4), new(8, 32, d=i8), new(8), new(4, 8)
    dy = new(4, 8, d=bf)
    bad = [lambda: I.gemm(x, sx, w, sw, y), lambda: I.gemm(q, None, w, sw, y), lambda: I.gemm(q, sx[:3], w, sw, y),
           lambda: I.gemm(x, None, w[:, :31], sw, y), lambda: I.gemm(x, None, x, sw, y), lambda: I.gemm(x, None, w, sw[:7], y),
           lambda: I.gemm(x, None, w, sw.double(), y), lambda: I.gemm(x, None, w, sw, y[:3]),
           lambda: I.gemm(x, None, w, sw, y[:, :7]), lambda: I.gemm(x, None, w, sw, y.double()),
           lambda: I.gemm(x, None, w, sw, y.cpu()), lambda: I.gemm(x, None, w.t().contiguous().t(), sw, y),
           lambda: I.gemm(x[0], None, w, sw, y), lambda: I.gemm(x[:1].expand(4, 32), None, w, sw, y),
           lambda: I.gemm(x, None, w, sw, y, workspace=new(3, d=torch.uint8)),
           lambda: I.gemm(x, None, w, sw, y, workspace=new(1 << 16)),
           lambda: I.gemm(new(1, I.MAX_COLS + 1), None, new(1, I.MAX_COLS + 1, d=i8), sw[:1], y[:1, :1]),
           lambda: I.gated(x, None, w, sw, w[:7], sw[:7], y), lambda: I.gated(x, None, w, sw, w, sw, y, "tanh"),
           lambda: I.quantize_rows(q, q, sx), lambda: I.quantize_rows(x, q[:, :31], sx), lambda: I.quantize_rows(x, q, sx[:2]),
           lambda: I.quantize_rows(x, x, sx),
           lambda: I.gemm_backward(dy.float(), q, sx, w, sw), lambda: I.gemm_backward(dy, x, None, w, sw),
           lambda: I.gemm_backward(dy[:, :7], q, sx, w, sw), lambda: I.gemm_backward(dy, q, sx, w, sw, x.half()),
           lambda: I.gemm_backward(dy, q, sx, w, sw, x[:3]), lambda: I.gemm_backward(dy, q, sx, w, sw, x, sw[:7]),
           lambda: I.gated_backward(dy, q, sx, w, sw, w, sw, x, sw, sw[:7]),
           lambda: I.gated_backward(dy, q, sx, w, sw, w, sw, x, activation=None),
           lambda: I.workspace_bytes("gated", x, None, w, sw), lambda: I.workspace_bytes("gemm_backward", q, sx, w, sw)]
    for f in bad:
        with pytest.raises(EntqError) as e:
            f()
        assert e.value.status == EINVAL
    # strided rows, a parameter's subclass and a one-row tensor of any stride pass
    I.gemm(torch.nn.Parameter(x, requires_grad=False), None, w, sw, y)
    I.gemm(new(4, 64, d=bf)[:, ::2][:, :0].reshape(4, 0), None, new(8, 0, d=i8), sw, y)
    I.gemm(new(9, 32, d=bf)[::9], None, w, sw, y[:1])
