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
