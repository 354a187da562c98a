"""GPU tests of the norms around a block against 64-bit references, at the
sizes, gates and values where they can go wrong."""
import numpy as np
import pytest
import torch

import norm_reference as R
from int8_reference import EPS

pytestmark = pytest.mark.gpu

KINDS = ("bf16", "f16", "f32")


@pytest.fixture(scope="module")
def N():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import entropy_coded_weight_amd as E
    E.lib()
    from entropy_coded_weight_amd import norm
    return norm


def matrix(m, n, kind, seed, pad=0, shift=0, size=1.0):
    """A matrix whose rows start at any element address (pad: between rows)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.full((m * (n + pad) + shift + 8,), 7.0, device="cuda").to(R.TYPES[kind])
    v = flat[shift:shift + m * (n + pad)].view(m, n + pad)[:, :n]
    v.copy_(size * torch.randn(m, n, device="cuda", generator=g))
    return v


def vector(n, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return 1 + 0.3 * torch.randn(n, device="cuda", generator=g)


def gate_of(which, m, n, kind, seed, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if which == "channel":
        return vector(n, seed) - 0.5
    if which == "token":
        return torch.randn(m, 1 + pad, device="cuda", generator=g)[:, :1]
    return matrix(m, n, kind, seed, pad, 1) if which == "full" else None


def close(got, want, bound, what):
    got = got.double()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs().max()), float((got - want)[bad][0]),
                           float(bound.expand_as(want)[bad][0]))


def codes_by_formula(s, pre):
    """numpy, by the stated fp32 arithmetic: codes and the scale before rho"""
    t = s.float().cpu().numpy() * pre.cpu().numpy()[None]
    top = np.abs(t).max(1, initial=0.0)
    c = np.maximum(top * np.float32(1 / 127), np.float32(2.0 ** -100)).astype(np.float32)
    inv = (np.float32(1) / c).astype(np.float32)
    return np.clip(np.rint((t * inv[:, None]).astype(np.float32)), -127, 127).astype(np.int8), c


SIZES = [(3, 1), (5, 7), (4, 64), (9, 255), (2, 512), (3, 513), (70, 2048), (3, 2049), (5, 4100), (2, 8192),
         (3, 8200), (2, 16384), (2, 16400), (1, 32768), (2, 40001)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", SIZES)
def test_forward(N, m, n, kind):
    for at, (gate, post, pad) in enumerate((("", False, 0), ("channel", True, 3), ("token", True, 8), ("full", True, 1),
                                            ("full", False, 0))):
        x, b = matrix(m, n, kind, at, pad, at), matrix(m, n, kind, 10 + at, pad, 3)
        w, pre = vector(n, 5) if post else None, vector(n, 6)
        g = gate_of(gate, m, n, kind, 7, pad)
        out, y = matrix(m, n, kind, 1, pad, 5), matrix(m, n, kind, 2, pad, 2)
        N.block(x, b, out, w, g, pre, y, alpha=0.75, beta=-1.5, eps=1e-5)
        want, bound = R.state(x, b, w, g, 0.75, -1.5, 1e-5, kind)
        close(out, want, bound, (gate, "out"))
        close(y, *R.normed(out, pre, 1e-5, kind), (gate, "y"))
        # the state alone, and its norm from the stored state: the same bits
        out2, y2 = torch.empty_like(out), torch.empty_like(y)
        N.block(x, b, out2, w, g, alpha=0.75, beta=-1.5, eps=1e-5)
        N.block(out, pre=pre, y=y2, eps=1e-5)
        assert torch.equal(out2, out) and torch.equal(y2, y)
        # codes
        q = torch.full((m, n + pad), 99, dtype=torch.int8, device="cuda")
        scale = torch.empty(m, device="cuda")
        N.block(x, b, out2, w, g, pre, q[:, :n], scale, alpha=0.75, beta=-1.5, eps=1e-5)
        assert torch.equal(out2, out) and bool((q[:, n:] == 99).all())
        codes, c = codes_by_formula(out, pre)
        assert np.array_equal(q[:, :n].cpu().numpy(), codes), gate
        want = torch.from_numpy(c).cuda().double() * R.rho(out.double(), 1e-5)[:, 0]
        close(scale, want, 3 * EPS * want, "scale")
        if pad:  # what lies between the rows stays
            tail = out.as_strided((m - 1, pad), (n + pad, 1), out.storage_offset() + n)
            assert bool((tail == 7).all())


BACK = [(1, 1), (5, 7), (4, 64), (9, 255), (2, 512), (3, 513), (70, 2048), (3, 2049), (5, 4100), (3, 8192), (3, 8200),
        (2, 16384), (2, 16400), (2, 40001), (1100, 96), (2600, 40), (600, 4096),
        (300, 4500)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", BACK)
def test_backward(N, m, n, kind):
    for at, (gate, post, pad) in enumerate((("", False, 0), ("", True, 2), ("channel", True, 3), ("token", True, 8),
                                            ("token", False, 0), ("full", True, 1), ("channel", False, 0))):
        s, b = matrix(m, n, kind, at, pad, at), matrix(m, n, kind, 10 + at, pad, 3)
        w, pre = vector(n, 5) if post else None, vector(n, 6)
        g = gate_of(gate, m, n, kind, 7, pad)
        dout, dy = matrix(m, n, kind, 20, pad, 1), matrix(m, n, kind, 21, pad, 6)
        dx, db = matrix(m, n, kind, 1, pad, 5), matrix(m, n, kind, 2, pad, 2)
        got = {"dx": dx, "dbranch": db, "dpre": torch.empty(n, device="cuda")}
        if post:
            got["dpost"] = torch.empty(n, device="cuda")
        if gate:
            got["dgate"] = gate_of(gate, m, n, kind, 8, pad)
        N.block_backward(s, dout, dy, b, w, g, pre, alpha=0.75, beta=-1.5, eps=1e-5, **got)
        want = R.gradients(s, dout, dy, b, w, g, pre, 0.75, -1.5, 1e-5, kind)
        assert set(got) == set(want)
        for name, v in got.items():
            close(v, *want[name], (gate, post, name))
        # each gradient alone, with the same bits
        for name, v in got.items():
            alone = torch.empty_like(v)
            N.block_backward(s, dout, dy, b, w, g, pre, alpha=0.75, beta=-1.5, eps=1e-5, **{name: alone})
            assert torch.equal(alone, v), (gate, post, name)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", [(3, 100), (2, 5000), (1030, 300), (2, 33000)])
def test_backward_of_one_incoming_gradient_or_no_branch(N, m, n, kind):
    s, b, d = matrix(m, n, kind, 1), matrix(m, n, kind, 2), matrix(m, n, kind, 3)
    w, pre, g = vector(n, 4), vector(n, 5), gate_of("token", m, n, kind, 6)
    new = lambda: torch.empty(m, n, dtype=s.dtype, device="cuda")  # noqa: E731
    vec = lambda: torch.empty(n, device="cuda")  # noqa: E731
    got = {"dx": new(), "dbranch": new(), "dpost": vec(), "dgate": torch.empty(m, 1, device="cuda")}
    N.block_backward(s, d, None, b, w, g, eps=1e-6, **got)
    want = R.gradients(s, d, None, b, w, g, None, 1, 1, 1e-6, kind)
    assert set(got) == set(want)
    for name, v in got.items():
        close(v, *want[name], name)
    got = {"dx": new(), "dbranch": new(), "dpost": vec(), "dpre": vec(), "dgate": torch.empty(m, 1, device="cuda")}
    N.block_backward(s, None, d, b, w, g, pre, beta=2.0, **got)
    want = R.gradients(s, None, d, b, w, g, pre, 1, 2.0, 1e-6, kind)
    for name, v in got.items():
        close(v, *want[name], name)
    got = {"dx": new(), "dpre": vec()}
    N.block_backward(s, d, d, pre=pre, **got)
    want = R.gradients(s, d, d, None, None, None, pre, 1, 1, 1e-6, kind)
    for name, v in got.items():
        close(v, *want[name], name)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n", [(1, 1), (5, 7), (3, 513), (3, 2049), (7, 4100), (3, 8192), (2, 8200), (600, 200)])
def test_backward_of_a_full_gate_without_norms(N, m, n, kind):
    """branch and gate alone (a sum of products), with either incoming gradient."""
    s, b, d, g = (matrix(m, n, kind, i, 1, i) for i in range(4))
    pre = vector(n, 5)
    for dy in (None, matrix(m, n, kind, 9)):
        got = {name: matrix(m, n, kind, 7, 2, 3) for name in ("dx", "dbranch", "dgate")}
        N.block_backward(s, d, dy, b, None, g, pre if dy is not None else None, alpha=-2.0, beta=0.5, **got)
        want = R.gradients(s, d, dy, b, None, g, pre, -2.0, 0.5, 1e-6, kind)
        for name, v in got.items():
            close(v, *want[name], name)
            tail = v.as_strided((m - 1, 2), (n + 2, 1), v.storage_offset() + n)
            assert bool((tail == 7).all()), name


@pytest.mark.parametrize("n", [24, 3000, 33000])
def test_large_and_small_values(N, n):
    """fp32 rows whose squares leave fp32's range; zero rows."""
    x = matrix(6, n, "f32", 1)
    x[1] *= 1e30
    x[2] *= 1e-25
    x[3] = 0
    x[4] *= 3e37
    pre, b = vector(n, 2), matrix(6, n, "f32", 3)
    b[5] *= 1e33
    b[0] = 0
    y, out = torch.empty_like(x), torch.empty_like(x)
    N.block(x, pre=pre, y=y, eps=1e-30)
    close(y, *R.normed(x, pre, 1e-30, "f32"), "y")
    N.block(x, b, out, pre, None, pre, y)
    close(out, *R.state(x, b, pre, None, 1, 1, 1e-6, "f32"), "out")
    d = matrix(6, n, "f32", 4)
    dx, db = torch.empty_like(x), torch.empty_like(x)
    N.block_backward(x, d, d, b, pre, None, pre, dx=dx, dbranch=db)
    want = R.gradients(x, d, d, b, pre, None, pre, 1, 1, 1e-6, "f32")
    close(dx, *want["dx"], "dx")
    close(db, *want["dbranch"], "dbranch")


@pytest.mark.parametrize("n", [40, 700, 9000, 40000])
@pytest.mark.parametrize("kind", KINDS)
def test_rows_that_are_not_finite(N, n, kind):
    """They stay in their rows: codes 0 of a NaN scale, NaN values."""
    x, pre = matrix(5, n, kind, 1), vector(n, 2)
    x[1, n // 2] = float("nan")
    x[2, 0] = float("inf")
    x[3, n - 1] = float("-inf")
    q, scale = torch.full((5, n), 9, dtype=torch.int8, device="cuda"), torch.empty(5, device="cuda")
    y = torch.empty_like(x)
    N.block(x, pre=pre, y=q, y_scales=scale)
    N.block(x, pre=pre, y=y)
    assert scale.isnan().tolist() == [False, True, True, True, False]
    assert (q[1:4] == 0).all() and (q[0] != 0).any() and (q[4] != 0).any()
    for r in (0, 4):
        close(y[r:r + 1], *R.normed(x[r:r + 1], pre, 1e-6, kind), "y")
    assert y[1].isnan().all() and y[2, 0].isnan() and (y[2, 1:] == 0).all() and (y[3, :-1] == 0).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [48, 5120, 33001])
def test_state_in_place(N, n, kind):
    x, b, w = matrix(7, n, kind, 1, 4, 1), matrix(7, n, kind, 2), vector(n, 3)
    out, y, y2 = (torch.empty(7, n, dtype=x.dtype, device="cuda") for _ in range(3))
    N.block(x, b, out, w, None, w, y, alpha=0.5)
    N.block(x, b, x, w, None, w, y2, alpha=0.5)
    assert torch.equal(x, out) and torch.equal(y, y2)


def test_rows_beyond_32_bits(N):
    """Row strides whose offsets, in elements and in bytes, pass 2^32."""
    n, ld = 700, 1_500_000_011
    room = torch.empty(3 * ld + 5000, dtype=torch.bfloat16, device="cuda")
    at = lambda i: room[i * 1000:].as_strided((4, n), (ld, 1))  # noqa: E731
    x, out, y = at(0), at(1), at(2)
    x.copy_(matrix(4, n, "bf16", 1))
    b, w = matrix(4, n, "bf16", 2), vector(n, 3)
    N.block(x, b, out, w, None, w, y)
    close(out, *R.state(x, b, w, None, 1, 1, 1e-6, "bf16"), "out")
    close(y, *R.normed(out, w, 1e-6, "bf16"), "y")
    dx, db, dpre = at(3), at(4), torch.empty(n, device="cuda")
    N.block_backward(out, y, b, b, w, None, w, dx, db, None, dpre)
    want = R.gradients(out, y, b, b, w, None, w, 1, 1, 1e-6, "bf16")
    for name, t in (("dx", dx), ("dbranch", db), ("dpre", dpre)):
        close(t, *want[name], name)


def test_empty(N):
    for m, n in ((0, 16), (3, 0), (0, 0)):
        x = torch.empty(m, n, device="cuda")
        w = torch.ones(n, device="cuda")
        N.block(x, x.clone(), x.clone(), w, None, w, x.clone())
        dpre, dpost, dg = torch.ones(n, device="cuda"), torch.ones(n, device="cuda"), torch.ones(n, device="cuda")
        N.block_backward(x, x, x, x, w, w, w, x.clone(), x.clone(), dg, dpre, dpost)
        assert not dpre.any() and not dpost.any() and not dg.any()
        dt = torch.ones(m, 1, device="cuda")
        if (m, n) != (0, 0):
            N.block_backward(x, x, x, x, w, torch.ones(m, 1, device="cuda"), w, dgate=dt)
            assert not dt.any()


def test_streams_and_graph(N):
    m, n = 130, 1032
    x, b, w = matrix(m, n, "bf16", 1), matrix(m, n, "bf16", 2), vector(n, 3)
    d = matrix(m, n, "bf16", 4)
    q, s, out = torch.empty(m, n, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda"), torch.empty_like(x)
    dx, db, dpre, dpost = torch.empty_like(x), torch.empty_like(x), torch.empty(n, device="cuda"), torch.empty(n, device="cuda")
    results = (q, s, out, dx, db, dpre, dpost)

    def run(stream=None):
        N.block(x, b, out, w, None, w, q, s, stream=stream)
        N.block_backward(out, d, d, b, w, None, w, dx, db, None, dpre, dpost, stream=stream)

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
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for k in range(4):
        x.copy_(matrix(m, n, "bf16", 50 + k))
        for t in results:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in results]
        run()
        assert all(torch.equal(a, t) for a, t in zip(results, got))


def test_refusals(N):
    import entropy_coded_weight_amd as E
    x, w = torch.ones(4, 32, device="cuda"), torch.ones(32, device="cuda")
    h, q, s = x.half(), torch.empty(4, 32, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    leaf = x.clone().requires_grad_()
    bad = [lambda: N.block(x, pre=w), lambda: N.block(x, y=x.clone()), lambda: N.block(x, x, pre=w, y=x.clone()),
           lambda: N.block(x, out=x.clone(), pre=w, y=x.clone()), lambda: N.block(x, post=w, pre=w, y=x.clone()),
           lambda: N.block(x, alpha=2, pre=w, y=x.clone()), lambda: N.block(x, h, x.clone()),
           lambda: N.block(x, x, h), lambda: N.block(x, pre=w, y=h), lambda: N.block(x, pre=w, y=q),
           lambda: N.block(x, pre=w, y=x.clone(), y_scales=s), lambda: N.block(x, pre=w, y=q, y_scales=s[:3]),
           lambda: N.block(x, pre=w[:31], y=x.clone()), lambda: N.block(x, pre=w.half(), y=x.clone()),
           lambda: N.block(x, x, x.clone(), gate=w[:5]), lambda: N.block(x, x, x.clone(), gate=torch.ones(1, 1, device="cuda").expand(4, 1)),
           lambda: N.block(x, x, x.clone(), gate=h), lambda: N.block(x, x[:3], x.clone()), lambda: N.block(x.t(), pre=s, y=x.t()),
           lambda: N.block(x, pre=w, y=x.clone(), eps=0.0), lambda: N.block(x, x, x.clone(), alpha=float("nan")),
           lambda: N.block(x, x, x.clone(), alpha="1"), lambda: N.block(leaf, pre=w, y=x.clone()),
           lambda: N.block(x, leaf, x.clone()), lambda: N.block(x, x, x.clone(), gate=leaf), lambda: N.block(x.double(), pre=w, y=x.double()),
           lambda: N.block_backward(x), lambda: N.block_backward(x, dy=x), lambda: N.block_backward(x, x, dpre=w),
           lambda: N.block_backward(x, x, dbranch=x.clone()), lambda: N.block_backward(x, x, branch=x, dpost=w),
           lambda: N.block_backward(x, x, branch=x, dgate=w), lambda: N.block_backward(x, leaf, dx=x.clone()),
           lambda: N.block_backward(x, x, branch=x, gate=w, dgate=torch.ones(4, 1, device="cuda")),
           lambda: N.block_backward(x, h, dx=x.clone()), lambda: N.block_backward(x, x, dx=h),
           lambda: N.block_backward(x, x, dx=x.clone(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))]
    for i, call in enumerate(bad):
        with pytest.raises(E.EntqError) as e:
            call()
        assert e.value.status == E.EINVAL, i
    ws = torch.empty(N.workspace_bytes(x, x, w, w, w), dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(x)
    N.block_backward(x, x, x, x, w, w, w, dx, workspace=ws)
