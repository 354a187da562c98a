"""CPU checks of the norms around a block: the gradient formulas against
central differences in 64 bits, and what the calls refuse before any launch
(through the binding and through the C interface)."""
import ctypes
import os

import pytest
import torch

import norm_reference as R


@pytest.fixture(scope="module")
def E():
    import entropy_coded_weight_amd as E
    if not os.path.exists(E.LIB_PATH):
        from entropy_coded_weight_amd import build
        build.build()
    return E


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", ["", "channel", "token", "full"])
def test_gradient_formulas_against_differences(gate, post):
    """L = sum(dout state) + sum(dy y) as a function of every input."""
    g = torch.Generator().manual_seed(3)
    m, n, alpha, beta, eps = 3, 5, 0.7, -1.3, 1e-2
    rand = lambda *s: torch.randn(*s, dtype=torch.float64, generator=g)  # noqa: E731
    args = {"dx": rand(m, n), "dbranch": rand(m, n), "dpre": rand(n)}
    if post:
        args["dpost"] = rand(n)
    if gate:
        args["dgate"] = rand(*{"channel": (n,), "token": (m, 1), "full": (m, n)}[gate])
    dout, dy = rand(m, n), rand(m, n)

    def forward(a):
        s, _ = R.state(a["dx"], a["dbranch"], a.get("dpost"), a.get("dgate"), alpha, beta, eps, "f32")
        return s, (dout * s).sum() + (dy * R.normed(s, a["dpre"], eps, "f32")[0]).sum()

    s, _ = forward(args)
    got = R.gradients(s, dout, dy, args["dbranch"], args.get("dpost"), args.get("dgate"), args["dpre"], alpha, beta,
                      eps, "f32")
    assert set(got) == set(args)
    e = 1e-5  # central differences: error of order e^2 and 1e-16 / e
    for name, (want, _) in got.items():
        for i in range(want.numel()):
            up, down = ({k: v.clone() for k, v in args.items()} for _ in range(2))
            up[name].view(-1)[i] += e
            down[name].view(-1)[i] -= e
            d = (forward(up)[1] - forward(down)[1]) / (2 * e)
            assert abs(d - want.reshape(-1)[i]) <= 1e-7 * (1 + want.abs().max()), (name, i)


def test_host_tensors_and_wrong_sets_of_arguments_are_refused(E):
    from entropy_coded_weight_amd import norm
    x, w = torch.zeros(2, 8), torch.ones(8)
    for call in (lambda: norm.block(x, pre=w, y=x), lambda: norm.block(None, pre=w, y=x),
                 lambda: norm.block_backward(x, x), lambda: norm.workspace_bytes(x)):
        with pytest.raises(E.EntqError, match="GPU") as e:
            call()
        assert e.value.status == E.EINVAL


# the C interface: addresses that are never dereferenced, since every call is
# refused (or empty) before a launch
A = 1 << 20
EALIGN, EWORKSPACE = -4, -5


def described(E, **k):
    f = dict(rows=4, cols=32, type=0, gate_kind=0, x=A, branch=A, gate=0, ldx=32, ldbranch=32, ldgate=32, post=A,
             pre=A, alpha=1.0, beta=1.0, eps=1e-6, reserved=0)
    f.update(k)
    return E.Norm(*f.values())


def forward(E, n=None, out=A, ldo=32, y=A, kind=0, ldy=32, scales=0):
    return E.lib().entq_norm_block(ctypes.byref(n) if n else None, out, ldo, y, kind, ldy, scales, None)


def backward(E, n=None, dout=A, lddo=32, dy=A, lddy=32, dx=A, lddx=32, db=A, lddb=32, dg=0, lddg=32, dpre=A, dpost=A,
             ws=A, room=1 << 40):
    return E.lib().entq_norm_block_backward(ctypes.byref(n) if n else None, dout, lddo, dy, lddy, dx, lddx, db, lddb,
                                            dg, lddg, dpre, dpost, ws, room, None)


@pytest.mark.parametrize("bad", [dict(type=3), dict(type=-1), dict(reserved=1), dict(cols=131072, ldx=131072),
                                 dict(rows=1 << 31), dict(eps=0.0), dict(eps=-1.0), dict(eps=float("inf")),
                                 dict(eps=float("nan")), dict(alpha=float("nan")), dict(beta=float("inf")),
                                 dict(x=0), dict(ldx=31), dict(ldbranch=31), dict(ldx=1 << 41), dict(gate_kind=4),
                                 dict(gate_kind=-1), dict(gate_kind=1), dict(gate=A), dict(branch=0),
                                 dict(branch=0, post=0, gate_kind=1, gate=A), dict(gate_kind=3, gate=A, ldgate=31),
                                 dict(gate_kind=2, gate=A, ldgate=0)])
def test_c_refuses_the_description(E, bad):
    n = described(E, **bad)
    assert forward(E, n) == E.EINVAL and backward(E, n) == E.EINVAL
    assert E.lib().entq_norm_block_backward_workspace_bytes(ctypes.byref(n)) == 0


@pytest.mark.parametrize("bad", [dict(x=A + 1), dict(branch=A + 1), dict(post=A + 2), dict(pre=A + 2),
                                 dict(type=2, x=A + 2), dict(gate_kind=3, gate=A + 1),
                                 dict(gate_kind=2, gate=A + 2), dict(gate_kind=1, gate=A + 2)])
def test_c_refuses_the_alignment(E, bad):
    n = described(E, **bad)
    assert forward(E, n) == EALIGN and backward(E, n) == EALIGN


def test_c_refusals_forward(E):
    n, bare = described(E), described(E, branch=0, post=0)
    assert forward(E, None) == E.EINVAL
    for k in (dict(out=0), dict(ldo=31), dict(ldy=31), dict(kind=2), dict(kind=7), dict(kind=3), dict(scales=A),
              dict(y=0, kind=3, scales=A)):
        assert forward(E, n, **k) == E.EINVAL, k
    assert forward(E, bare) == E.EINVAL  # a state without a branch
    assert forward(E, bare, out=0, y=0) == E.EINVAL
    assert forward(E, described(E, pre=0)) == E.EINVAL
    for k in (dict(out=A + 1), dict(y=A + 1), dict(kind=3, scales=A + 2)):
        assert forward(E, n, **k) == EALIGN, k
    assert forward(E, described(E, rows=0)) == 0
    assert forward(E, described(E, cols=0, x=0, branch=0, post=0, pre=0), out=0, y=0) == 0


def test_c_refusals_backward(E):
    n, bare = described(E), described(E, branch=0, post=0)
    assert backward(E, None) == E.EINVAL
    for k in (dict(dout=0, dy=0, dpre=0), dict(lddo=31), dict(lddy=31), dict(lddx=31), dict(lddb=31), dict(dg=A),
              dict(dy=0)):
        assert backward(E, n, **k) == E.EINVAL, k
    assert backward(E, bare) == E.EINVAL and backward(E, bare, db=0) == E.EINVAL
    assert backward(E, described(E, pre=0)) == E.EINVAL
    full = described(E, gate_kind=3, gate=A)
    assert backward(E, full, dg=A, lddg=31) == E.EINVAL
    assert backward(E, described(E, gate_kind=2, gate=A), dg=A, lddg=0) == E.EINVAL
    for k in (dict(dout=A + 1), dict(dy=A + 1), dict(dx=A + 1), dict(db=A + 1), dict(dpre=A + 2), dict(dpost=A + 1),
              dict(ws=A + 128)):
        assert backward(E, n, **k) == EALIGN, k
    assert backward(E, full, dg=A + 1) == EALIGN
    need = E.lib().entq_norm_block_backward_workspace_bytes(ctypes.byref(n))
    assert need > 0
    assert backward(E, n, room=need - 1) == EWORKSPACE and backward(E, n, ws=0) == EWORKSPACE
