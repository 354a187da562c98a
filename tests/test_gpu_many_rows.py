"""GPU tests of more rows than one launch of the norms and the distillation
takes (2^20 workgroups, of up to four rows)."""
import pytest
import torch

import distill_reference
import norm_reference

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


@pytest.fixture(scope="module")
def E():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import entropy_coded_weight_amd as E
    E.lib()
    return E


@pytest.mark.parametrize("m,n", [((1 << 22) + 5, 3), ((1 << 20) + 3, 260)])
def test_norms(E, m, n):
    """Against 64 bits: the sum, its inverse root (1 ulp) and two products."""
    from entropy_coded_weight_amd import norm
    g = torch.Generator(device="cuda").manual_seed(n)
    x, w = torch.randn(m, n, device="cuda", generator=g), 1 + 0.2 * torch.randn(n, device="cuda", generator=g)
    y = torch.full_like(x, 7.0)
    norm.block(x, pre=w, y=y, eps=1e-5)
    rho = norm_reference.rho(x.double(), 1e-5)
    want = x.double() * rho * w.double()
    assert bool(((y.double() - want).abs() <= 4 * EPS * want.abs() + 2.0 ** -149).all())
    codes, scales = torch.empty(m, n, dtype=torch.int8, device="cuda"), torch.empty(m, device="cuda")
    norm.block(x, pre=w, y=codes, y_scales=scales, eps=1e-5)
    t = x * w
    c = t.abs().amax(1) * torch.tensor(1 / 127, device="cuda")
    assert bool((codes == (t * torch.reciprocal(c)[:, None]).round().to(torch.int8)).all())
    assert bool(((scales.double() - c.double() * rho[:, 0]).abs() <= 3 * EPS * scales.double()).all())
    # the gradient: of all rows' state, and of pre over all of them
    dx, dw = torch.empty_like(x), torch.empty(n, device="cuda")
    norm.block_backward(x, dy=y, pre=w, dx=dx, dpre=dw, eps=1e-5)
    u, dy = x.double() * rho, y.double()
    v = dy * w.double()
    mean = (u * v).mean(1, keepdim=True)
    size = rho * (v.abs() + u.abs() * mean.abs())
    assert bool(((dx.double() - rho * (v - u * mean)).abs() <= 8 * EPS * size + 2.0 ** -149).all())
    terms = dy * u
    # (fp32 over a strip of rows, at least 256 strips)
    assert bool(((dw.double() - terms.sum(0)).abs() <= (m / 256 + 8) * EPS * terms.abs().sum(0)).all())


def test_distillation(E):
    from entropy_coded_weight_amd import distill
    m, v, k = (1 << 20) + 7, 9, 2
    g = torch.Generator(device="cuda").manual_seed(3)
    z = torch.randn(m, v, device="cuda", generator=g)
    teacher, index = torch.topk(z + 0.5 * torch.randn(m, v, device="cuda", generator=g), k, dim=1)
    lse = torch.logsumexp(teacher, 1) + 0.3
    loss, grad = torch.full((m,), 7.0, device="cuda"), torch.full_like(z, 7.0)
    distill.loss_backward(z, index, teacher, grad, None, loss, lse)
    want = distill_reference.distill(z, index, teacher, lse)
    for got, (value, bound) in ((loss, want[0]), (grad, want[1])):
        assert bool(((got.double() - value).abs() <= bound).all())
