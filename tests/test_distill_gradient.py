"""CPU checks of the distillation's reference where the teacher's masses do not
sum to 1: its gradient against autograd of its own loss in 64 bits."""
import pytest
import torch

import distill_reference as R


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("v,k", [(9, 3), (5, 9), (6, 6), (40, 12)])
def test_gradient_against_autograd(v, k, tail):
    """Rows of masses above 1 (a lse too low, a teacher rounded to 16 bits, a
    class with two entries) and below (a lse too high; entries of every class)."""
    g = torch.Generator().manual_seed(10 * v + k)
    m = 7
    full = 2 * torch.randn(m, v, dtype=torch.float64, generator=g)
    full[:, 0] += 4
    z = (full + 0.5 * torch.randn(m, v, dtype=torch.float64, generator=g)).requires_grad_()
    teacher, index = torch.topk(full, min(k, v), dim=1)
    if k > v:
        index, teacher = torch.cat([index, index[:, :k - v]], 1), torch.cat([teacher, teacher[:, :k - v]], 1)
    index[3, 1:] = -1
    index[4, 1] = index[4, 0]
    teacher[5] = teacher[5].bfloat16().double()
    lse = torch.logsumexp(full / 1.25, 1) + torch.tensor([0.3, -0.3, 1e-3, -1e-3, 0.0, 0.0, -2.0]) if tail else None
    dloss = torch.tensor([1.0, -2.0, 0.5, 3.0, 1.0, 1.0, 1.0])
    (loss, _), (got, bound) = R.distill(z, index, teacher, lse, None, 1.25, dloss)
    want = torch.autograd.grad((loss * dloss).sum(), z)[0]
    # (sums of some v terms in 64 bits, each of a few roundings)
    size = dloss.abs()[:, None] * (1 + torch.softmax(z.detach() / 1.25, 1)) * (8 if tail else 1)
    assert ((got - want).abs() <= 64 * v * 2.0 ** -53 * size).all()
    assert (got.sum(1).abs() <= 64 * v * 2.0 ** -53 * size.sum(1)).all()
    assert (bound > 0).all()


def test_more_mass_than_one():
    """The example by hand: the only likely class, mass 1.051. The stated loss has
    a gradient of 4e-5 there and not q - p = -0.05."""
    z = torch.tensor([[20.0, 8.0, 7.0]], dtype=torch.float64)
    lse = torch.logsumexp(torch.tensor([[19.95, 9.0, 8.0]], dtype=torch.float64), 1)
    index, teacher = torch.tensor([[0]]), torch.tensor([[20.0]])
    p, q = float(torch.exp(20.0 - lse)), float(torch.softmax(z, 1)[0, 0])
    assert p > 1.05
    (loss, _), (g, _) = R.distill(z, index, teacher, lse)
    assert abs(float(loss) - p * (float(torch.log(torch.tensor(p, dtype=torch.float64)))
                                  - float(torch.log_softmax(z, 1)[0, 0]))) < 1e-12
    assert abs(float(g[0, 0]) - (p * q - p)) < 1e-14 and -1e-4 < float(g[0, 0]) < 0
    assert abs(float(g.sum())) < 1e-14
