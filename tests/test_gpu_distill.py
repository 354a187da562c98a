"""GPU tests of the distillation loss and its gradient against 64-bit
references."""
import pytest
import torch

import distill_reference as R
from norm_reference import TYPES

pytestmark = pytest.mark.gpu

KINDS = ("bf16", "f16", "f32")


@pytest.fixture(scope="module")
def D():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import entropy_coded_weight_amd as E
    E.lib()
    from entropy_coded_weight_amd import distill
    return distill


def inputs(m, v, k, kind, seed, tail, wide=False, pad=0, teacher_kind="f32", missing=False, weights=False, spread=2.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    full = spread * torch.randn(m, v, device="cuda", generator=g)
    full[:, :min(8, v)] += 4 * torch.rand(m, min(8, v), device="cuda", generator=g)
    teacher, index = torch.topk(full, min(k, v), dim=1)
    if k > v:  # entries of one class twice
        more = torch.randint(0, v, (m, k - v), device="cuda", generator=g)
        index, teacher = torch.cat([index, more], 1), torch.cat([teacher, full.gather(1, more)], 1)
    lse = torch.logsumexp(full / 1.25, 1) if tail else None
    if missing:
        index = torch.where(torch.rand(index.shape, device="cuda", generator=g) < 0.3, -1, index)
        index[m // 2] = -3
    flat = torch.full((m, v + pad), 5.0, device="cuda").to(TYPES[kind])
    logits = flat[:, pad // 2:pad // 2 + v]
    logits.copy_(full + 0.8 * torch.randn(m, v, device="cuda", generator=g))
    table = torch.zeros(m, k + pad, dtype=torch.int64 if wide else torch.int32, device="cuda")
    table[:, :k] = index
    w = None
    if weights:
        w = torch.rand(m, device="cuda", generator=g) - 0.25
        w[::3] = 0
    return logits, table[:, :k], teacher.to(TYPES[teacher_kind]), lse, w


def close(got, want, bound, what):
    got = got.double()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs().max()), float((got - want)[bad][0]),
                           float(bound.expand_as(want)[bad][0]))


def check(D, logits, index, teacher, lse, weight, kind, T=1.25, dloss=None, grad_kind=None):
    m, v = logits.shape
    grad_kind = grad_kind or kind
    loss, again = torch.full((m,), 9.0, device="cuda"), torch.full((m,), 9.0, device="cuda")
    flat = torch.full((m, v + 3), 7.0, device="cuda").to(TYPES[grad_kind])
    grad = flat[:, 1:v + 1]
    D.loss(logits, index, teacher, loss, lse, weight, T)
    D.loss_backward(logits, index, teacher, grad, dloss, again, lse, weight, T)
    want = R.distill(logits, index, teacher, lse, weight, T, dloss, grad_kind)
    close(loss, *want[0], "loss")
    close(again, *want[0], "loss beside the gradient")
    close(grad, *want[1], "gradient")
    assert bool((flat[:, 0] == 7).all()) and bool((flat[:, v + 1:] == 7).all())
    return loss, grad


SIZES = [(3, 1, 1), (2, 5, 9), (5, 64, 3), (9, 1000, 64), (3, 4097, 100), (7, 8191, 256), (3, 8192, 1), (2, 8200, 33),
         (6, 32000, 64), (2, 32768, 20), (2, 40000, 8), (2, 50021, 65), (2, 65537, 7), (1, 131072, 200), (2, 262144, 4)]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,v,k", SIZES)
def test_loss_and_gradient(D, m, v, k, kind):
    for at, (tail, wide, pad, tk, missing, weights) in enumerate((
            (False, False, 0, "f32", False, False), (True, True, 0, "bf16", False, True),
            (True, False, 6, "f32", True, False), (False, True, 3, "f16", True, True))):
        logits, index, teacher, lse, w = inputs(m, v, k, kind, at, tail, wide, pad, tk, missing, weights)
        dloss = torch.linspace(-2, 1, m, device="cuda") if at % 2 else None
        check(D, logits, index, teacher, lse, w, kind, dloss=dloss)


@pytest.mark.parametrize("grad_kind", ["bf16", "f16"])
@pytest.mark.parametrize("v", [7, 1001, 9000, 33001, 70003])
def test_16_bit_gradients_of_fp32_logits(D, v, grad_kind):
    for tail in (False, True):
        logits, index, teacher, lse, w = inputs(4, v, 12, "f32", 3, tail, missing=True, weights=True)
        check(D, logits, index, teacher, lse, w, "f32", grad_kind=grad_kind)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("v", [200, 9000])
def test_a_sure_student_and_a_sure_teacher(D, v, kind):
    """The mass outside the entries far below fp32's resolution of 1 on either
    side, and a class whose probability is 0."""
    logits, index, teacher, lse, _ = inputs(6, v, 8, kind, 3, True)
    logits[0, index[0].long()] += 40
    logits[1, index[1].long()] -= 60
    teacher[2, 0] += 30
    lse[2] = torch.logsumexp(teacher[2] / 1.25, 0)
    teacher[3, 1] = -float("inf")
    other = [c for c in range(v) if c not in index[4].tolist()][:3]
    logits[4, other] = -float("inf")
    check(D, logits, index, teacher, lse, None, kind)
    check(D, logits, index, teacher, None, None, kind)
    # no probability where the teacher has some: an infinite loss, a finite gradient
    logits[5, int(index[5, 2])] = -float("inf")
    loss, grad = torch.empty(6, device="cuda"), torch.empty_like(logits)
    for rest in (lse, None):
        D.loss_backward(logits, index, teacher, grad, None, loss, rest, None, 1.25)
        assert torch.isinf(loss[5]) and loss[5] > 0 and torch.isfinite(loss[:5]).all() and torch.isfinite(grad).all()


def test_entries_that_cover_every_class(D):
    """There is no tail then, whatever the rounding of the teacher's sum."""
    logits, index, teacher, lse, _ = inputs(4, 60, 60, "f32", 1, True)
    check(D, logits, index, teacher, lse + 1e-3, None, "f32")


def test_large_logits(D):
    logits, index, teacher, lse, _ = inputs(4, 5000, 16, "f32", 1, True)
    logits[1] += 1e4
    logits[2] *= 1e5
    logits[3] -= 3e4
    # (their exponents are differences of logits: exact up to the logits' own steps)
    check(D, logits, index, teacher, lse, None, "f32")
    check(D, logits, index, teacher, None, None, "f32", T=1.0)


@pytest.mark.parametrize("v", [300, 9000, 33000, 60000, 150000])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("kind", KINDS)
def test_masks_of_the_lowest_value(D, v, tail, kind):
    """Rows of which a mask of the type's lowest value, or of -inf, leaves some
    classes, one, or none; rows of large logits of either sign. Differences of
    logits are what counts: the reference's are exact in 64 bits."""
    logits, index, teacher, lse, _ = inputs(8, v, 8, kind, 4, tail)
    low = torch.finfo(logits.dtype).min
    logits[1, v // 3:] = low
    logits[2] = low                                     # nothing left: all alike
    logits[3] = low
    logits[3, index[3, 0].long()] = 1.5
    logits[4] = -logits[4].abs() * (3e4 if kind != "f16" else 3e3)
    logits[5, 7:] = float("-inf")
    index[5] = torch.arange(8, dtype=torch.int32, device="cuda") % 7
    logits[6] = float("-inf")
    logits[6, index[6].long()] = 0.5 * teacher[6].to(logits.dtype)
    logits[7] = -low
    logits[7, 3] = low
    index[7] = torch.arange(10, 18, dtype=torch.int32, device="cuda")
    if tail:
        lse[2] = lse[3] = torch.logsumexp(teacher[2].double() / 1.25, 0).float() + 3
        teacher[3] = teacher[2]
    T = 1.25
    loss, grad = torch.empty(8, device="cuda"), torch.empty_like(logits)
    D.loss_backward(logits, index, teacher, grad, None, loss, lse, None, T)
    # in 64 bits from each row's largest
    z = logits.double()
    z = (z - z.amax(1, keepdim=True)) / T
    want = R.distill(z * T, index, teacher, lse, None, T, None, kind)
    ok = [0, 1, 2, 4, 7]
    assert torch.isfinite(want[0][0][ok]).all()
    close(loss[ok], want[0][0][ok], want[0][1][ok], "loss")
    close(grad[ok], want[1][0][ok], want[1][1][ok], "gradient")
    assert loss[5:7].isinf().tolist() == want[0][0][5:7].isinf().tolist()  # (what the student rules out)
    for r in (5, 6):
        if torch.isfinite(want[1][0][r]).all():
            close(grad[r:r + 1], want[1][0][r:r + 1], want[1][1][r:r + 1], r)
    # row 3's classes outside the entries are alike, and far from the one that is
    # left: 64 bits hold no 2.7e38 + log v, so its gradient is written out here
    hit = torch.zeros(v, dtype=torch.bool, device="cuda").scatter_(0, index[3].long(), True)
    p = torch.exp(teacher[3].double() / T - lse[3].double()) if tail else torch.softmax(teacher[3].double() / T, 0)
    g = torch.full((v,), -(1 - float(p.sum())) / (v - int(hit.sum())) if tail else 0.0, dtype=torch.float64, device="cuda")
    g[index[3].long()] = -p
    g[index[3, 0].long()] += 1
    g = g / T
    close(grad[3], g, (R.ROUND[kind] + 64 * R.EPS) * g.abs() + 64 * R.EPS * hit + R.TINY[kind], "gradient of row 3")


@pytest.mark.parametrize("v", [300, 33000, 150000])
@pytest.mark.parametrize("tail", [False, True])
def test_masked_and_broken_rows(D, v, tail):
    nan = float("nan")
    logits, index, teacher, lse, _ = inputs(7, v, 8, "bf16", 4, tail)
    w = torch.ones(7, device="cuda")
    keep = logits.clone()
    logits[1] = nan
    logits[2, 7] = float("inf")
    w[1] = w[2] = 0
    teacher[2] = nan
    index[3] = -1
    logits[3, 5] = nan
    index[4, 2] = v       # no such class
    index[5, 0] = 2 ** 31 - 1
    logits[6, 123] = nan
    loss, grad = torch.empty(7, device="cuda"), torch.empty_like(logits)
    D.loss_backward(logits, index, teacher, grad, None, loss, lse, w, 1.25)
    assert loss.isnan().tolist() == [False, False, False, False, True, True, True]
    assert loss[1:4].tolist() == [0, 0, 0] and not grad[1:4].any()
    assert grad[4:].isnan().all()
    want = R.distill(keep[:1], index[:1], teacher[:1], None if lse is None else lse[:1], None, 1.25, None, "bf16")
    close(loss[:1], *want[0], "loss")
    close(grad[:1], *want[1], "gradient")


def test_rows_beyond_32_bits(D):
    """Row strides whose offsets, in elements and in bytes, pass 2^32."""
    v, ld = 3001, 1_500_000_011
    logits, index, teacher, lse, _ = inputs(4, v, 9, "f16", 6, True)
    room = torch.empty(3 * ld + 4 * v, dtype=torch.float16, device="cuda")
    far, grad = room.as_strided((4, v), (ld, 1)), room[2 * v:].as_strided((4, v), (ld, 1))
    far.copy_(logits)
    loss = torch.empty(4, device="cuda")
    D.loss_backward(far, index, teacher, grad, None, loss, lse, None, 1.25)
    want = R.distill(logits, index, teacher, lse, None, 1.25, None, "f16")
    close(loss, *want[0], "loss")
    close(grad, *want[1], "gradient")


def test_empty(D):
    x = torch.empty(0, 10, device="cuda")
    D.loss(x, torch.empty(0, 3, dtype=torch.int64, device="cuda"), torch.empty(0, 3, device="cuda"), torch.empty(0, device="cuda"))
    D.loss_backward(x, torch.empty(0, 3, dtype=torch.int64, device="cuda"), torch.empty(0, 3, device="cuda"), x.clone())


def test_streams_and_graph(D):
    logits, index, teacher, lse, w = inputs(40, 9001, 20, "bf16", 5, True, weights=True)
    loss, alone, grad = torch.empty(40, device="cuda"), torch.empty(40, device="cuda"), torch.empty_like(logits)
    results = (loss, alone, grad)

    def run(stream=None):
        D.loss(logits, index, teacher, alone, lse, w, 1.25, stream)
        D.loss_backward(logits, index, teacher, grad, None, loss, lse, w, 1.25, stream)

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
        logits.copy_(inputs(40, 9001, 20, "bf16", 60 + k, True)[0])
        for t in results:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in results]
        run()
        assert all(torch.equal(a, t) for a, t in zip(results, got))


def test_refusals(D):
    import entropy_coded_weight_amd as E
    x, i = torch.zeros(4, 50, device="cuda"), torch.zeros(4, 6, dtype=torch.int64, device="cuda")
    t, out = torch.zeros(4, 6, device="cuda"), torch.zeros(4, device="cuda")
    leaf = x.clone().requires_grad_()
    bad = [lambda: D.loss(leaf, i, t, out), lambda: D.loss(x.double(), i, t, out), lambda: D.loss(x, i.short(), t, out),
           lambda: D.loss(x, i[:, :5], t, out), lambda: D.loss(x, i[:3], t, out), lambda: D.loss(x, i, t[:3], out),
           lambda: D.loss(x, i.t().contiguous().t(), t, out), lambda: D.loss(x, i.cpu(), t, out), lambda: D.loss(x, i, t, out[:3]),
           lambda: D.loss(x, i, t, out.half()), lambda: D.loss(x, i, t, out, teacher_lse=out[:2]),
           lambda: D.loss(x, i, t, out, weight=out.double()), lambda: D.loss(x, i, t, out, temperature=0),
           lambda: D.loss(x, i, t, out, temperature=float("nan")), lambda: D.loss(x, i, t, out, temperature=2e4),
           lambda: D.loss(x, i.repeat(1, 50), t.repeat(1, 50), out), lambda: D.loss(x[:, :0], i, t, out),
           lambda: D.loss(x, i, t.int(), out), lambda: D.loss(torch.zeros(1, 262145, device="cuda"), i[:1], t[:1], out[:1]),
           lambda: D.loss_backward(x.half(), i, t, x.clone()), lambda: D.loss_backward(x, i, t, x.double()), lambda: D.loss_backward(x, i, t, x[:, :49]),
           lambda: D.loss_backward(x, i, t, x.clone(), dloss=out[:1]), lambda: D.loss(x, i, t[0], out)]
    for n, call in enumerate(bad):
        with pytest.raises(E.EntqError) as e:
            call()
        assert e.value.status == E.EINVAL, n
