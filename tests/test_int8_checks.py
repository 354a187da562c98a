"""CPU checks of the int8 products: the gradient formulas against central
differences in 64 bits, and what the calls refuse before any launch (through
the binding and through the C interface)."""
import ctypes
import os

import numpy as np
import pytest
import torch

import int8_reference as R


@pytest.fixture(scope="module")
def E():
    import entropy_coded_weight_amd as E
    if not os.path.exists(E.LIB_PATH):
        from entropy_coded_weight_amd import build
        build.build()
    return E


@pytest.fixture(scope="module")
def I(E):
    from entropy_coded_weight_amd import int8
    return int8


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gradient_formulas_against_differences(name):
    """L = sum(dh * H) as a function of the dequantised activations and of
    each channel scale."""
    rng = np.random.default_rng(4)
    m, n, k = 3, 5, 4
    q = rng.integers(-9, 10, (m, k)).astype(np.int8)
    sx = np.full(m, 0.1)
    wg, wu = (rng.integers(-9, 10, (n, k)).astype(np.int8) for _ in range(2))
    sg, su = rng.uniform(0.1, 0.4, n), rng.uniform(-0.4, -0.1, n)
    dh = rng.standard_normal((m, n))

    def loss(x, sg, su):  # x: the activations the codes stand for
        g, u = x @ wg.T.astype(float) * sg, x @ wu.T.astype(float) * su
        return (dh * R.act(name, g)[0].numpy() * u).sum()

    x = q * sx[:, None]
    (dx, _), (dsg, _), (dsu, _) = R.gated_backward(dh, q, sx, wg, sg, wu, su, name, "bf16")
    e = 1e-5  # central differences: error of order e^2 and 1e-16 / e
    for want, at in ((dx.numpy(), 0), (dsg.numpy(), 1), (dsu.numpy(), 2)):
        args = [x, sg, su]
        for i in np.ndindex(want.shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[at][i] += e
            down[at][i] -= e
            d = (loss(*up) - loss(*down)) / (2 * e)
            assert abs(d - want[i]) <= 1e-7 * (1 + abs(want).max()), (at, i)


def test_plain_product_gradient_against_differences():
    rng = np.random.default_rng(5)
    m, n, k = 3, 4, 5
    q, w = rng.integers(-9, 10, (m, k)).astype(np.int8), rng.integers(-9, 10, (n, k)).astype(np.int8)
    sx, sw, dy = rng.uniform(0.1, 1, m), rng.uniform(-1, 1, n), rng.standard_normal((m, n))
    (dx, _), (ds, _) = R.gemm_backward(dy, q, sx, w, sw, "f16")
    dx, ds = dx.numpy(), ds.numpy()
    loss = lambda x, s: (dy * (x @ w.T.astype(float) * s)).sum()  # noqa: E731
    x = q * sx[:, None]
    for i in np.ndindex(dx.shape):
        step = np.zeros_like(x)
        step[i] = 1e-4  # linear: differences are exact to rounding
        assert abs((loss(x + step, sw) - loss(x - step, sw)) / 2e-4 - dx[i]) < 1e-9
    for i in range(n):
        step = np.zeros(n)
        step[i] = 1e-4
        assert abs((loss(x, sw + step) - loss(x, sw - step)) / 2e-4 - ds[i]) < 1e-9


def test_quantizer_reference_values():
    q, s = R.quantize(np.array([[127.0, -1.0, 0.5, 1.5, 2.5], [0, 0, 0, 0, 0], [np.nan, 1, 2, 3, 4]], np.float32))
    assert s[0] == np.float32(127 * np.float32(1 / 127)) and s[1] == np.float32(2.0 ** -100) and np.isnan(s[2])
    assert q.tolist() == [[127, -1, 0, 2, 2], [0] * 5, [0] * 5]


def test_host_tensors_are_refused(E, I):
    x, w, s = torch.zeros(2, 16), torch.zeros(3, 16, dtype=torch.int8), torch.ones(3)
    y = torch.zeros(2, 3)
    q, sx = torch.zeros(2, 16, dtype=torch.int8), torch.ones(2)
    for call in (lambda: I.gemm(x, None, w, s, y), lambda: I.quantize_rows(x, q, sx),
                 lambda: I.gated(x, None, w, s, w, s, y), lambda: I.gemm_backward(y.half(), q, sx, w, s),
                 lambda: I.gated_backward(y.half(), q, sx, w, s, w, s), lambda: I.gemm(None, None, w, s, y),
                 lambda: I.workspace_bytes("gemm", x, None, w, s)):
        with pytest.raises(E.EntqError, match="GPU") as e:
            call()
        assert e.value.status == E.EINVAL
    with pytest.raises(E.EntqError, match="workspace_bytes of 'product'"):
        I.workspace_bytes("product", x, None, w, s)


# the C interface: addresses that are never dereferenced, since every call is
# refused (or empty) before a launch
A = 1 << 20


def rows(E, r, c, kind=3, ld=None, data=A, scales=A, reserved=0):
    return E.Rows(data, c if ld is None else ld, scales if kind == 3 else 0, r, c, kind, reserved)


def forward(E, I, x=None, w=None, up=None, y=A, kind=0, ldy=None, act=0, ws=A, ws_bytes=1 << 40):
    x = x or rows(E, 4, 32)
    w = w or rows(E, 8, 32)
    ldy = w.rows if ldy is None else ldy
    b = ctypes.byref
    if up is None:
        return E.lib().entq_int8_gemm(b(x), b(w), y, kind, ldy, ws, ws_bytes, None)
    return E.lib().entq_int8_gated(b(x), b(w), b(up), act, y, kind, ldy, ws, ws_bytes, None)


EALIGN, EWORKSPACE = -4, -5


def test_c_refusals_forward(E, I):
    bad = [dict(x=rows(E, 4, 31)), dict(x=rows(E, 4, 32, ld=31)), dict(x=rows(E, 4, 32, data=0)),
           dict(x=rows(E, 4, 32, scales=0)), dict(x=rows(E, 4, 32, kind=4)), dict(x=rows(E, 4, 32, kind=-1)),
           dict(x=rows(E, 4, 32, reserved=1)), dict(w=rows(E, 8, 32, kind=0)), dict(w=rows(E, 8, 32, scales=0)),
           dict(w=rows(E, 8, 32, ld=1 << 41)), dict(y=0), dict(kind=3), dict(kind=7), dict(ldy=7),
           dict(x=rows(E, 4, 131072), w=rows(E, 8, 131072)), dict(x=rows(E, 1 << 31, 32)),
           dict(up=rows(E, 7, 32)), dict(up=rows(E, 8, 32, kind=2)), dict(up=rows(E, 8, 33)),
           dict(up=rows(E, 8, 32), act=4), dict(up=rows(E, 8, 32), act=-1)]
    for k in bad:
        assert forward(E, I, **k) == E.EINVAL, {n: getattr(v, "cols", v) for n, v in k.items()}
    x = E.Rows(A, 32, A, 4, 32, 0, 0)  # activations with scales
    assert forward(E, I, x=x) == E.EINVAL
    L, b = E.lib(), ctypes.byref
    assert L.entq_int8_gemm(None, b(rows(E, 8, 32)), A, 0, 8, A, 1 << 40, None) == E.EINVAL
    assert L.entq_int8_gemm(b(rows(E, 8, 32)), None, A, 0, 8, A, 1 << 40, None) == E.EINVAL
    for k in (dict(y=A + 1), dict(y=A + 2, kind=2), dict(x=rows(E, 4, 32, scales=A + 2)),
              dict(x=rows(E, 4, 32, kind=0, data=A + 1)), dict(x=rows(E, 4, 32, kind=2, data=A + 2)),
              dict(x=rows(E, 4, 32, kind=0), ws=A + 128)):
        assert forward(E, I, **k) == EALIGN
    act = rows(E, 4, 32, kind=0)
    need = E.lib().entq_int8_gemm_workspace_bytes(b(act), b(rows(E, 8, 32)))
    assert need > 0
    assert forward(E, I, x=act, ws_bytes=need - 1) == EWORKSPACE
    assert forward(E, I, x=act, ws=0, ws_bytes=0) == EWORKSPACE
    assert E.lib().entq_int8_gemm_workspace_bytes(b(act), b(rows(E, 8, 33))) == 0
    assert E.lib().entq_int8_gemm_workspace_bytes(None, None) == 0


def test_c_refusals_backward(E, I):
    L, b = E.lib(), ctypes.byref
    x, w, dy = rows(E, 4, 32), rows(E, 8, 32), rows(E, 4, 8, kind=0)

    def back(dy=dy, x=x, w=w, dx=A, lddx=32, ds=A, ws=A, n=1 << 40):
        return L.entq_int8_gemm_backward(dy and b(dy), x and b(x), w and b(w), dx, lddx, ds, ws, n, None)

    def gated(dy=dy, up=w, act=0, dx=A, lddx=32, ds=A, du=A, ws=A, n=1 << 40):
        return L.entq_int8_gated_backward(dy and b(dy), b(x), b(w), up and b(up), act, dx, lddx, ds, du, ws, n, None)

    for k in (dict(dy=rows(E, 4, 9, kind=0)), dict(dy=rows(E, 5, 8, kind=0)), dict(dy=rows(E, 4, 8, kind=2)),
              dict(dy=rows(E, 4, 8)), dict(dy=rows(E, 4, 8, kind=0, ld=7)), dict(dy=rows(E, 4, 8, kind=0, data=0)),
              dict(dy=None), dict(lddx=31)):
        assert back(**k) == E.EINVAL, k
        assert gated(**k) == E.EINVAL, k
    assert back(x=rows(E, 4, 32, kind=0)) == E.EINVAL
    assert gated(act=9) == E.EINVAL and gated(up=rows(E, 9, 32)) == E.EINVAL and gated(up=None) == E.EINVAL
    for k in (dict(dx=A + 1), dict(ds=A + 2), dict(ws=A + 64), dict(dy=rows(E, 4, 8, kind=1, data=A + 1))):
        assert back(**k) == EALIGN and gated(**k) == EALIGN, k
    assert gated(du=A + 1) == EALIGN
    assert back(n=255) == EWORKSPACE and gated(ws=0) == EWORKSPACE
    assert back(dx=0, ds=0) == E.lib().entq_int8_gemm_backward(b(dy), b(x), b(w), 0, 32, 0, A, 1 << 40, None) == 0


def test_c_refusals_quantize(E, I):
    L, b = E.lib(), ctypes.byref
    for r, q, ld, s, want in ((rows(E, 4, 32), A, 32, A, E.EINVAL), (rows(E, 4, 32, kind=0), A, 31, A, E.EINVAL),
                              (rows(E, 4, 32, kind=0), 0, 32, A, E.EINVAL),
                              (rows(E, 4, 32, kind=0), A, 32, 0, E.EINVAL),
                              (rows(E, 4, 32, kind=0), A, 32, A + 1, EALIGN),
                              (rows(E, 4, 131072, kind=0), A, 131072, A, E.EINVAL),
                              (rows(E, 0, 32, kind=0), 0, 32, 0, 0)):
        assert L.entq_quantize_rows(b(r), q, ld, s, None) == want
    assert L.entq_quantize_rows(None, A, 32, A, None) == E.EINVAL
