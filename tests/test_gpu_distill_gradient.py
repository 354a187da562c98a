"""GPU tests of the distillation gradient where the teacher's mass is not 1 or
not a number, where it nearly cancels, and where it is very small."""
import pytest
import torch

import distill_reference as R
from norm_reference import TYPES
from test_gpu_distill import D, KINDS, close, inputs  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("v", [300, 5000, 33000, 150000])
@pytest.mark.parametrize("tail", [False, True])
def test_a_nan_of_the_teacher_reaches_every_class(D, v, tail):  # noqa: F811
    """A NaN among the entries' logits (one that is no entry's does not count),
    or in place of their log-sum."""
    logits, index, teacher, lse, _ = inputs(5, v, 8, "bf16", 4, tail)
    keep = [t.clone() if t is not None else None for t in (logits, index, teacher, lse)]
    teacher[1, 3] = float("nan")
    index[2, 5] = -1
    teacher[2, 5] = float("nan")
    index[4] = -1
    if tail:
        lse[3] = lse[4] = float("nan")
    else:
        teacher[3] = float("nan")
    loss, grad = torch.empty(5, device="cuda"), torch.empty_like(logits)
    D.loss_backward(logits, index, teacher, grad, None, loss, lse, None, 1.25)
    assert loss.isnan().tolist() == [False, True, False, True, False]
    assert grad[1].isnan().all() and grad[3].isnan().all()
    assert loss[4] == 0 and not grad[4].any()
    want = R.distill(*(t[:1] if t is not None else None for t in keep), None, 1.25, None, "bf16")
    close(loss[:1], *want[0], "loss")
    close(grad[:1], *want[1], "gradient")
    assert torch.isfinite(loss[2]) and torch.isfinite(grad[2]).all()


def exact(logits, index, teacher, lse, weight, T, dloss=None):
    """Loss and gradient by autograd in 64 bits, from the loss's definition."""
    T = float(torch.tensor(T, dtype=torch.float32))
    z = (logits.double() / T).requires_grad_()
    inside, at = index >= 0, index.clamp_min(0).long()
    t = torch.where(inside, teacher.double() / T, -float("inf"))
    logp = torch.log_softmax(t, 1) if lse is None else t - lse.double()[:, None]
    p = torch.where(inside, logp.exp(), 0)
    L = torch.logsumexp(z, 1)
    loss = torch.where(p > 0, p * (torch.where(p > 0, logp, 0) - z.gather(1, at) + L[:, None]), 0).sum(1)
    if lse is not None:
        hit = torch.zeros_like(z).detach().scatter_add_(1, at, inside.double()) > 0
        pt = torch.where(hit.all(1), 0, (1 - p.sum(1)).clamp_min(0))
        Lt = torch.logsumexp(z.masked_fill(hit, -float("inf")), 1)
        loss = loss + torch.where(pt > 0, pt * (pt.clamp_min(1e-300).log() - Lt + L), 0)
    if weight is not None:
        loss = loss * weight.double()
    by = torch.ones_like(loss) if dloss is None else dloss.double()
    return loss.detach(), torch.autograd.grad((loss * by).sum(), z)[0] / T


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("v", [64, 1001, 9000, 33001, 150000])
def test_a_mass_that_is_not_one(D, v, kind):  # noqa: F811
    """The teacher's masses sum to more than 1, or the entries cover every class
    and sum to less: L counts with their sum."""
    logits, index, teacher, lse, _ = inputs(6, v, 20, kind, 7, True)
    teacher[0] += 0.05                          # as 16-bit logits beside the sum of the unrounded ones
    teacher[0, 0] += 9
    logits[0, int(index[0, 0])] += 9
    lse[0] = torch.logsumexp(teacher[0].double() / 1.25, 0).float() - 0.05
    index[1, 10:] = index[1, :10].clone()       # every entry twice
    teacher[1, 10:] = teacher[1, :10].clone()
    lse[1] = torch.logsumexp(teacher[1].double() / 1.25, 0).float() - 0.3
    lse[2] = torch.logsumexp(teacher[2].double() / 1.25, 0).float() - 1e-3
    lse[3] -= 4
    dloss = torch.tensor([1.0, -2.0, 0.5, 3.0, 1.0, 1.0], device="cuda")
    sets = [(logits, index, teacher, lse)]
    if v == 64:
        all_, every = inputs(6, v, v, kind, 8, True)[:4], torch.tensor([1e-3, -1e-3, 0.4, -0.4, 0.0, 2.0], device="cuda")
        sets.append((*all_[:3], all_[3] + every))
    for logits, index, teacher, lse in sets:
        for t in (teacher, teacher.bfloat16()):
            loss, grad = torch.empty(6, device="cuda"), torch.empty_like(logits)
            D.loss_backward(logits, index, t, grad, dloss, loss, lse, None, 1.25)
            want = exact(logits, index, t, lse, None, 1.25, dloss)
            bounds = R.distill(logits, index, t, lse, None, 1.25, dloss, kind)
            close(loss, want[0], bounds[0][1], "loss")
            close(grad, want[1], bounds[1][1], "gradient")
            # L moves all logits alike: a row's gradients sum to 0
            assert (grad.double().sum(1).abs() <= bounds[1][1].sum(1)).all()


@pytest.mark.parametrize("v", [60, 1001, 20000, 33001, 60000, 150000])
@pytest.mark.parametrize("near", [1e-2, 1e-4, -1e-5])
def test_the_tail_of_student_and_teacher_alike(D, v, near):  # noqa: F811
    """qt - pt far below both. The classes outside the entries have the logit 0,
    so that their powers and the sum of these are exact in fp32, and what is
    left of the arithmetic is that in 64 bits (1e-14 of qt, 1e-9 of the
    factor) and roundings to fp32: of a gradient outside the factor's and the
    product's, of the entries' the result's; four are allowed."""
    torch.manual_seed(v)
    T, k = 1.25, 8
    logits = torch.zeros(4, v, device="cuda")
    index = torch.stack([torch.randperm(v, device="cuda")[:k] for _ in range(4)])
    top = T * torch.log(torch.tensor(v / k, device="cuda")) + torch.tensor([0.0, 1.0, -2.0, 3.0], device="cuda")[:, None]
    logits.scatter_(1, index, (top + 0.5 * torch.randn(4, k, device="cuda")).clamp_min(0.01))
    z = logits.double() / T
    # the student's own masses, a constant below or above in the logarithm
    L = torch.logsumexp(z, 1)
    inside = torch.exp(z - L[:, None]).gather(1, index).sum(1)
    lse = (L - torch.log1p(-near * (1 - inside) / inside)).float()
    teacher = logits.gather(1, index)
    loss, grad = torch.empty(4, device="cuda"), torch.empty_like(logits)
    D.loss_backward(logits, index, teacher, grad, None, loss, lse, None, T)
    p = torch.exp(teacher.double() / T - lse.double()[:, None])
    hit = torch.zeros_like(logits, dtype=torch.bool).scatter_(1, index, True)
    share = (v - k) * torch.ones(4, dtype=torch.float64, device="cuda")
    # (torch's softmax of 64 bits is off by 5e-7 of its values on this GPU)
    q = torch.exp(z - L[:, None])
    factor = share / torch.exp(L) - (1 - p.sum(1))
    want = torch.where(hit, q, (factor / share)[:, None])
    want.scatter_add_(1, index, -p)
    size = torch.where(hit, q, want.abs())
    size.scatter_add_(1, index, p)
    slack = 1e-14 / torch.exp(L)[:, None]
    close(grad, want / T, (4 * R.EPS * size + slack) / T + R.TINY["f32"], "gradient")
    # (that far apart, and what rounding lse moves sum p by)
    assert (factor.abs() <= 1.02 * abs(near) * (1 - p.sum(1)) + 1.02 * R.EPS * lse.double().abs()).all()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v", [700, 9001, 33001, 150000])
@pytest.mark.parametrize("by", [1e-14, 1e-22, 1e-30, 1e30])
def test_very_small_and_large_weights(D, v, tail, by):  # noqa: F811
    """Gradients far from 1 in size are as exact as others while fp32 holds them."""
    logits, index, teacher, lse, _ = inputs(4, v, 12, "f32", 5, tail)
    dloss = torch.tensor([1.0, -0.3, 2.0, 0.7], device="cuda") * by
    grad = torch.empty_like(logits)
    D.loss_backward(logits, index, teacher, grad, dloss, None, lse, None, 1.25)
    _, (want, bound) = R.distill(logits, index, teacher, lse, None, 1.25, dloss, "f32")
    close(grad, want, bound, "gradient")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("v", [500, 9000, 33001, 150000, 262144])
@pytest.mark.parametrize("power", [-3, 0, 2])
def test_small_losses_at_the_stated_error(D, v, power, kind):  # noqa: F811
    """A loss of 1e-4 to 0.7 against the bound of the exponents' rounded factor
    alone, |scale / (log2(e) / T) - 1| E_q |z - max|, and the result's rounding:
    T is log2(e) times a power of two and the logits multiples of it, so that
    every exponent is a whole number, every power and sum exact in fp32."""
    T = float(torch.tensor(1.44269504088896340736 * 2.0 ** power, dtype=torch.float32))
    scale64 = 1.44269504088896340736 / T
    scale = float(torch.tensor(scale64, dtype=torch.float32))
    assert scale == 2.0 ** -power
    m = 4
    steps = torch.tensor([22, 21, 20, 18], device="cuda")   # (a thread's sum with the largest: within 2^-23 .. 2^9)
    logits = (-steps[:, None] * 2.0 ** power).repeat(1, v).to(TYPES[kind])
    index = torch.tensor([[3], [v - 1], [v // 2], [7]], device="cuda")
    logits.scatter_(1, index, 0.0)
    loss, alone, grad = torch.empty(m, device="cuda"), torch.empty(m, device="cuda"), torch.empty_like(logits)
    D.loss(logits, index, torch.zeros(m, 1, device="cuda"), alone, temperature=T)
    D.loss_backward(logits, index, torch.zeros(m, 1, device="cuda"), grad, None, loss, temperature=T)
    z = logits.double() / T
    rest = (v - 1) * torch.exp(z.min(1).values)             # the sum is 1 + this
    want = torch.log1p(rest)
    slope = abs(scale / scale64 - 1) * (rest / (1 + rest)) * z.min(1).values.abs()
    bound = 1.001 * slope + R.EPS * want + 1e-12 * want
    close(loss, want, bound, "loss beside the gradient")
    close(alone, want, bound, "loss")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("v", [40, 5000, 33000, 150000])
@pytest.mark.parametrize("tail", [False, True])
def test_a_row_of_minus_infinity_alone(D, v, tail, kind):  # noqa: F811
    """There is no softmax of it: NaN, and not 0 for the classes outside."""
    logits, index, teacher, lse, _ = inputs(4, v, 8, kind, 4, tail)
    logits[1:3] = -float("inf")
    index[2] = -1
    loss, grad = torch.empty(4, device="cuda"), torch.empty_like(logits)
    D.loss_backward(logits, index, teacher, grad, None, loss, lse, None, 1.25)
    assert loss.isnan().tolist() == [False, True, False, False]
    assert grad[1].isnan().all() and torch.isfinite(grad[[0, 3]]).all()
    assert loss[2] == 0 and not grad[2].any()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("v", [40, 5000, 33000, 150000])
@pytest.mark.parametrize("tail", [False, True])
def test_no_number_among_the_students_logits(D, v, tail, kind):  # noqa: F811
    """A NaN or an infinity at an entry's class and at another: no softmax of the
    row, whatever the entry's mass is."""
    logits, index, teacher, lse, _ = inputs(6, v, 8, kind, 4, tail)
    other = next(c for c in range(v) if c not in index[1:5].flatten().tolist())
    logits[1, int(index[1, 0])] = float("nan")
    logits[2, other] = float("nan")
    logits[3, int(index[3, 0])] = float("inf")
    logits[4, other] = float("inf")
    logits[5, int(index[5, 2])] = float("nan")
    teacher[5, 2] = -float("inf")
    loss, grad = torch.empty(6, device="cuda"), torch.empty_like(logits)
    D.loss_backward(logits, index, teacher, grad, None, loss, lse, None, 1.25)
    assert loss.isnan().tolist() == [False] + [True] * 5
    assert grad[1:].isnan().all() and torch.isfinite(grad[0]).all()


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v", [300, 9000, 150000])
def test_entries_of_masses_below_fp32(D, v, tail):  # noqa: F811
    """Masses below fp32's smallest number, times a weight that brings them back."""
    logits, index, teacher, lse, _ = inputs(3, v, 8, "f32", 6, tail)
    at = index[:, 5:].long()
    low = logits.amax(1, keepdim=True) - 1.25 * torch.tensor([[106.0, 112.0, 118.0]], device="cuda")
    logits.scatter_(1, at, low)
    teacher[:, 5:] = teacher[:, :1] - 1.25 * torch.tensor([[107.0, 111.5, 119.0]], device="cuda")
    dloss = torch.tensor([1e30, -3e28, 2e32], device="cuda")
    grad = torch.empty_like(logits)
    D.loss_backward(logits, index, teacher, grad, dloss, None, lse, None, 1.25)
    _, (want, bound) = R.distill(logits, index, teacher, lse, None, 1.25, dloss, "f32")
    assert bool((want.gather(1, at) != 0).all())
    close(grad, want, bound, "gradient")
