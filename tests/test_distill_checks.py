"""CPU checks of the distillation loss: its gradient formula against central
differences in 64 bits, and what the calls refuse before any launch."""
import ctypes
import os

import pytest
import torch

import distill_reference as R


@pytest.fixture(scope="module")
def E():
    import entropy_coded_weight_amd as E
    if not os.path.exists(E.LIB_PATH):
        from entropy_coded_weight_amd import build
        build.build()
    return E


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_against_differences(tail):
    g = torch.Generator().manual_seed(2)
    m, v, k = 4, 9, 3
    z = torch.randn(m, v, dtype=torch.float64, generator=g)
    full = 2 * torch.randn(m, v, dtype=torch.float64, generator=g)
    teacher, index = torch.topk(full, k, dim=1)
    index[1, 2] = -1
    index[2] = -1
    index[3, 1] = index[3, 0]  # one class twice
    lse = torch.logsumexp(full / 1.5, 1) + 0.4 if tail else None
    weight = torch.tensor([1.0, 0.5, 2.0, -1.5])
    dloss = torch.tensor([1.0, -2.0, 1.0, 0.25])
    run = lambda x: R.distill(x, index, teacher, lse, weight, 1.5, dloss)  # noqa: E731
    (loss, _), (grad, _) = run(z)
    assert loss[2] == 0 and not grad[2].any() and (loss[:2] > 0).all()
    e = 1e-5  # central differences: error of order e^2 and 1e-16 / e
    for i in range(z.numel()):
        up, down = z.clone(), z.clone()
        up.view(-1)[i] += e
        down.view(-1)[i] -= e
        d = ((run(up)[0][0] - run(down)[0][0]) * dloss).sum() / (2 * e)
        assert abs(d - grad.view(-1)[i]) < 1e-8


def test_teacher_equal_to_student_has_no_loss():
    z = torch.randn(3, 20, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    t, i = torch.topk(z, 5, dim=1)
    (loss, _), (g, _) = R.distill(z, i, t, torch.logsumexp(z, 1))
    assert loss.abs().max() < 1e-14 and g.abs().max() < 1e-14


def test_host_tensors_are_refused(E):
    from entropy_coded_weight_amd import distill
    x, i, t, out = torch.zeros(2, 9), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 3), torch.zeros(2)
    for call in (lambda: distill.loss(x, i, t, out), lambda: distill.loss_backward(x, i, t, x), lambda: distill.loss(None, i, t, out)):
        with pytest.raises(E.EntqError, match="GPU") as e:
            call()
        assert e.value.status == E.EINVAL


# the C interface: addresses that are never dereferenced, since every call is
# refused (or empty) before a launch
A = 1 << 20
EALIGN = -4


def described(E, **k):
    f = dict(rows=4, classes=100, top=8, type=0, teacher_type=2, index_bytes=4, temperature=1.0, reserved=0, logits=A,
             index=A, teacher=A, ldlogits=100, ldindex=8, ldteacher=8, lse=0, weight=0)
    f.update(k)
    return E.Distill(*f.values())


def loss(E, d, out=A):
    return E.lib().entq_distill_loss(ctypes.byref(d) if d else None, out, None)


def back(E, d, dloss=0, dl=A, kind=0, ld=100, out=0):
    return E.lib().entq_distill_backward(ctypes.byref(d) if d else None, dloss, dl, kind, ld, out, None)


@pytest.mark.parametrize("bad", [dict(reserved=1), dict(type=3), dict(type=-1), dict(teacher_type=3), dict(index_bytes=2),
                                 dict(rows=1 << 31), dict(classes=0), dict(classes=262145, ldlogits=262145), dict(top=0),
                                 dict(top=257, ldindex=257, ldteacher=257), dict(ldlogits=99), dict(ldindex=7),
                                 dict(ldteacher=7), dict(ldlogits=1 << 41), dict(temperature=0.0), dict(temperature=-1.0),
                                 dict(temperature=float("nan")), dict(temperature=float("inf")), dict(temperature=1e-5),
                                 dict(temperature=1e5), dict(logits=0), dict(index=0), dict(teacher=0)])
def test_c_refuses_the_description(E, bad):
    d = described(E, **bad)
    assert loss(E, d) == E.EINVAL and back(E, d) == E.EINVAL


def test_c_refusals(E):
    d = described(E)
    assert loss(E, None) == E.EINVAL and back(E, None) == E.EINVAL
    assert loss(E, d, 0) == E.EINVAL and back(E, d, dl=0) == E.EINVAL and back(E, d, ld=99) == E.EINVAL
    for kind in (1, 2, 3, -1):
        assert back(E, d, kind=kind) == E.EINVAL
    assert back(E, described(E, type=2), kind=3) == E.EINVAL
    assert loss(E, d, A + 2) == EALIGN
    for k in (dict(dl=A + 1), dict(dloss=A + 1), dict(out=A + 2)):
        assert back(E, d, **k) == EALIGN
    for k in (dict(logits=A + 1), dict(teacher=A + 2), dict(index=A + 2), dict(index=A + 4, index_bytes=8), dict(lse=A + 1),
              dict(weight=A + 2)):
        bad = described(E, **k)
        assert loss(E, bad) == EALIGN and back(E, bad) == EALIGN, k
    none = described(E, rows=0, logits=0, index=0, teacher=0)
    assert loss(E, none, 0) == 0 and back(E, none, dl=0) == 0
