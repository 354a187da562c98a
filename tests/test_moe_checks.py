"""CPU checks of the mixture-of-experts layer: its reference against the
feed-forward formulas token by token, and what the calls refuse before any
launch."""
import ctypes
import os

import numpy as np
import pytest
import torch

import int8_reference as I
import moe_reference as R


@pytest.fixture(scope="module")
def E():
    import entropy_coded_weight_amd as E
    if not os.path.exists(E.LIB_PATH):
        from entropy_coded_weight_amd import build
        build.build()
    return E


def test_reference_token_by_token():
    g = torch.Generator().manual_seed(1)
    m, e, k, d, f, n = 5, 4, 2, 12, 7, 6
    codes = lambda *s: torch.randint(-9, 10, s, generator=g, dtype=torch.int8)  # noqa: E731
    scale = lambda *s: 0.1 + torch.rand(*s, generator=g)  # noqa: E731
    x, router = torch.randn(m, d, generator=g), torch.randn(e, d, generator=g)
    w = [codes(e, f, d), scale(e, f), codes(e, f, d), scale(e, f), codes(e, n, f), scale(e, n)]
    at, p, y, bound = R.layer(x, router, *w, k, "gelu", True, "f32")
    assert torch.allclose(p.sum(1), torch.ones(m, dtype=torch.float64))
    q, sx = I.quantize(x.numpy())
    for t in range(m):
        logits = (router.double() @ x[t].double()).tolist()
        best = sorted(range(e), key=lambda i: (-logits[i], i))[:k]
        assert at[t].tolist() == best
        soft = np.exp(np.array([logits[i] for i in best]))
        want = np.zeros(n)
        for i, s in zip(best, soft / soft.sum()):
            h, _ = I.gated(q[t:t + 1], sx[t:t + 1], w[0][i], w[1][i], w[2][i], w[3][i], "gelu")
            qh, sh = I.quantize(h.numpy())
            want += s * (qh[0].astype(float) @ w[4][i].double().numpy().T) * sh[0] * w[5][i].double().numpy()
        assert (np.abs(want - y[t].numpy()) <= bound[t].numpy()).all()


def test_ties_go_to_the_lowest_index():
    x, router = torch.ones(1, 3), torch.tensor([[0.0, 0, 1], [1, 0, 0], [0, 1, 0], [2, -1, 0]])
    assert R.choose(x, router, 3, True)[0].tolist() == [[0, 1, 2]]


def test_host_tensors_are_refused(E):
    from entropy_coded_weight_amd import moe
    x, r, w = torch.zeros(2, 8), torch.zeros(3, 8), torch.zeros(3, 8, 8, dtype=torch.int8)
    s = torch.ones(3, 8)
    for call in (lambda: moe.few(x, r, w, s, w, s, w, s, x, 1), lambda: moe.workspace_bytes(x, r, w, s, w, s, w, s, 1)):
        with pytest.raises(E.EntqError, match="GPU") as e:
            call()
        assert e.value.status == E.EINVAL


# the C interface: addresses that are never dereferenced, since every call is
# refused (or empty) before a launch
A = 1 << 20
EALIGN, EWORKSPACE = -4, -5


def tokens(E, **k):
    f = dict(data=A, ld=32, scales=0, rows=4, cols=32, type=0, reserved=0)
    f.update(k)
    return E.Rows(*f.values())


def experts(E, **k):
    f = dict(experts=8, top_k=2, hidden=48, out=40, activation=0, normalize=1, router_type=2, reserved=0, router=A,
             ldrouter=32, weights=[A, A, A], scales=[A, A, A], ld=[32, 32, 48], stride=[48 * 32, 48 * 32, 48 * 40],
             scale_stride=[48, 48, 40])
    f.update(k)
    v = list(f.values())
    return E.Experts(*v[:10], (ctypes.c_void_p * 3)(*v[10]), (ctypes.c_void_p * 3)(*v[11]), *((ctypes.c_uint64 * 3)(*a) for a in v[12:]))


def call(E, x=None, e=None, y=A, kind=0, ldy=40, chosen=0, p=0, ws=A, room=1 << 40):
    x, e = x or tokens(E), e or experts(E)
    return E.lib().entq_moe_few(ctypes.byref(x), ctypes.byref(e), y, kind, ldy, chosen, p, ws, room, None)


@pytest.mark.parametrize("bad", [dict(rows=65), dict(type=3), dict(type=-1), dict(scales=A), dict(reserved=1), dict(cols=0),
                                 dict(cols=33), dict(ld=31), dict(data=0), dict(ld=1 << 41)])
def test_c_refuses_the_tokens(E, bad):
    assert call(E, tokens(E, **bad)) == E.EINVAL
    assert E.lib().entq_moe_few_workspace_bytes(ctypes.byref(tokens(E, **bad)), ctypes.byref(experts(E))) == 0


@pytest.mark.parametrize("bad", [dict(experts=0), dict(experts=257), dict(top_k=0), dict(top_k=9), dict(hidden=0), dict(out=0),
                                 dict(hidden=131072), dict(out=(1 << 22) + 1), dict(activation=4), dict(activation=-1),
                                 dict(normalize=2), dict(router_type=3), dict(reserved=1), dict(router=0), dict(ldrouter=31),
                                 dict(weights=[A, 0, A]), dict(scales=[A, A, 0]), dict(ld=[32, 31, 48]), dict(ld=[32, 32, 47]),
                                 dict(stride=[48 * 32, 48 * 32 - 1, 48 * 40]), dict(stride=[48 * 32, 1 << 41, 48 * 40]),
                                 dict(scale_stride=[48, 48, 39]), dict(experts=40, top_k=33)])
def test_c_refuses_the_experts(E, bad):
    assert call(E, e=experts(E, **bad)) == E.EINVAL
    assert E.lib().entq_moe_few_workspace_bytes(ctypes.byref(tokens(E)), ctypes.byref(experts(E, **bad))) == 0


def test_c_refusals(E):
    b, L = ctypes.byref, E.lib()
    assert L.entq_moe_few(None, b(experts(E)), A, 0, 40, 0, 0, A, 1 << 40, None) == E.EINVAL
    assert L.entq_moe_few(b(tokens(E)), None, A, 0, 40, 0, 0, A, 1 << 40, None) == E.EINVAL
    for k in (dict(y=0), dict(kind=3), dict(kind=-1), dict(ldy=39), dict(ldy=1 << 41)):
        assert call(E, **k) == E.EINVAL, k
    for k in (dict(y=A + 1), dict(kind=2, y=A + 2), dict(chosen=A + 2), dict(p=A + 1), dict(ws=A + 128)):
        assert call(E, **k) == EALIGN, k
    assert call(E, tokens(E, data=A + 1)) == EALIGN and call(E, e=experts(E, router=A + 2)) == EALIGN
    assert call(E, e=experts(E, scales=[A, A + 2, A])) == EALIGN
    need = L.entq_moe_few_workspace_bytes(b(tokens(E)), b(experts(E)))
    assert need > 0
    assert call(E, room=need - 1) == EWORKSPACE and call(E, ws=0) == EWORKSPACE
    assert call(E, tokens(E, rows=0, data=0), y=0) == 0
