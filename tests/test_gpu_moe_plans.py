"""GPU tests of the plans that a mixture of experts takes: where its tensors
and their scales may lie."""
import pytest
import torch

from test_gpu_moe import E, M, plan_of  # noqa: F401

pytestmark = pytest.mark.gpu


def moved(E, b, out=None, scales=None):  # noqa: F811
    t = b.tensors.copy()
    if out is not None:
        t["out_elem_offset"] = out
    if scales is not None:
        t["scale_row_offset"] = scales
    return E.plan(t, b.freq, b.chunks, b.blob.size)


def test_experts_that_share_scales_or_lie_backwards_are_refused(E, M):  # noqa: F811
    """One set of scales for all experts (a plan may say so), or experts from the
    buffer's end down: no step between experts, which the layer needs."""
    e, d, f, n = 3, 64, 32, 48
    b, p, blob, scales, w = plan_of(E, e, d, f, n)
    router = torch.randn(e, d, device="cuda")
    at, rows = [int(v) for v in b.tensors["out_elem_offset"]], [int(v) for v in b.tensors["scale_row_offset"]]
    back = lambda v: [v[3 * (e - 1 - i // 3) + i % 3] for i in range(3 * e)]  # noqa: E731
    for out, own in ((None, rows[:3] * e), (back(at), None), (None, back(rows)), (back(at), back(rows))):
        q = moved(E, b, out, own)
        with pytest.raises(E.EntqError) as ei:
            M.MixtureOfExperts(q, torch.ones(4 * scales.numel(), device="cuda"), router, 1)
        assert ei.value.status == E.EINVAL


def test_gaps_between_experts(E, M):  # noqa: F811
    e, d, f, n, m = 3, 64, 32, 48, 5
    b, p, blob, scales, w = plan_of(E, e, d, f, n)
    torch.manual_seed(2)
    x, router = torch.randn(m, d, device="cuda"), torch.randn(e, d, device="cuda")
    want, y = torch.empty(m, n, device="cuda"), torch.empty(m, n, device="cuda")
    M.few(x, router, *w, want, 2)
    out = [int(v) + 160 * (i // 3) for i, v in enumerate(b.tensors["out_elem_offset"])]
    rows = [int(v) + 7 * (i // 3) for i, v in enumerate(b.tensors["scale_row_offset"])]
    q = moved(E, b, out, rows)
    spread = torch.full((q.scale_rows,), float("nan"), device="cuda")
    for i in range(e):
        spread[rows[3 * i]:rows[3 * i] + 2 * f + n] = scales[i * (2 * f + n):(i + 1) * (2 * f + n)]
    mix = M.MixtureOfExperts(q, spread, router, 2)
    mix.decode(blob)
    mix.forward(x, y)
    assert torch.equal(y, want)


def test_what_is_no_activation_is_refused(E, M):  # noqa: F811
    b, p, blob, scales, w = plan_of(E, 2, 64, 32, 48)
    mix = M.MixtureOfExperts(p, scales, torch.zeros(2, 64, device="cuda"), 1)
    y = torch.zeros(3, 48, device="cuda")
    for x in (None, 3.0, [[0.0] * 64], torch.zeros(3, 64), torch.zeros(64, device="cuda"), torch.zeros(3, 63, device="cuda"),
              torch.zeros(3, 64, dtype=torch.int8, device="cuda"), torch.zeros(1, 3, 64, device="cuda")):
        with pytest.raises(E.EntqError) as ei:
            mix.forward(x, y)
        assert ei.value.status == E.EINVAL
    x = torch.zeros(3, 64, device="cuda")
    for bad in (dict(y=None), dict(experts=[1]), dict(weights=3)):
        with pytest.raises(E.EntqError) as ei:
            mix.forward(x, **{"y": y, **bad})
        assert ei.value.status == E.EINVAL
