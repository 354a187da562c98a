"""The RMS norms before and after a block with its gate and residual scale
(the entq_norm_* calls of include/entq.h): what stands between two blocks of a
transformer in one pass over its rows. With rho(v) = 1 / sqrt(mean(v^2) + eps),

    state = alpha x + beta gate v,   v = branch rho(branch) post   (branch without post)
    y     = state rho(state) pre

x is the residual, branch a block's output; y goes to the next block, in the
activations' type or as the int8 codes and scales that ``int8.gemm`` and
``int8.gated`` take, which saves the quantiser's pass.

Matrices are bfloat16, float16 or float32 [M, N], all of one type (unit stride
along N, any row stride and alignment); post and pre float32 [N]; gate a
factor per channel (float32 [N]), per token (float32 [M, 1]) or per value (the
matrices' type, [M, N]). Streams, workspaces, and what needs an autograd graph
are as in ``int8``; post, pre and gates of float32 may be parameters, whose
gradients the backward call writes.
"""
from __future__ import annotations

import math

import torch

from . import EINVAL, EntqError, Norm, lib
from .int8 import (_BF16, _F16, _F32, _I8, MAX_COLS, _enqueue, _gpu, _matrix, _no_graph, _vector)

_NONE, _CHANNEL, _TOKEN, _FULL = 0, 1, 2, 3
_FLOATS = (_BF16, _F16, _F32)


def _number(name, v):
    if type(v) is float and -3e38 <= v <= 3e38:
        return v
    if not isinstance(v, (int, float)) or not math.isfinite(v) or abs(v) > 3e38:
        raise EntqError(EINVAL, f"{name} is {v!r}: a finite number is required")
    return float(v)


def _gate(name, t, kind, index, m, n):
    """(entq_gate, row stride) of a factor or of its gradient for matrices of
    type ``kind``."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise EntqError(EINVAL, f"{name}: a torch tensor on cuda:{index} is required")
    if t.dim() == 1:
        _vector(name, t, index, n)
        return _CHANNEL, n
    if t.dtype == torch.float32 and t.shape == (m, 1) and (n != 1 or kind != _F32):
        # (any stride along the tokens, but not one value for all)
        if m > 1 and t.stride(0) < 1:
            raise EntqError(EINVAL, f"{name}: strides {t.stride()}; a value of its own for each "
                                    "token is required")
        return _TOKEN, max(1, t.stride(0))
    return _FULL, _matrix(name, t, index, (kind,), (m, n))[1]


def _describe(x, branch, post, gate, pre, alpha, beta, eps, what="x"):
    index = _gpu(what, x)
    kind, ldx = _matrix(what, x, index, _FLOATS)
    _no_graph(what, x)
    m, n = shape = x.shape
    if n > MAX_COLS:
        raise EntqError(EINVAL, f"{what} has {n} columns, at most {MAX_COLS} are taken")
    b = p = g = w = 0
    ldb = ldg = n
    gate_kind = _NONE
    if branch is not None:
        _, ldb = _matrix("branch", branch, index, (kind,), shape)
        _no_graph("branch", branch)
        b = branch.data_ptr()
    elif post is not None or gate is not None or alpha != 1 or beta != 1:
        raise EntqError(EINVAL, "post, gate, alpha and beta belong to a branch")
    if post is not None:
        p = _vector("post", post, index, n)
    if pre is not None:
        w = _vector("pre", pre, index, n)
    if gate is not None:
        gate_kind, ldg = _gate("gate", gate, kind, index, m, n)
        if gate_kind == _FULL:
            _no_graph("gate", gate)
        g = gate.data_ptr()
    a = Norm(m, n, kind, gate_kind, x.data_ptr(), b, g, ldx, ldb, ldg, p, w,
             _number("alpha", alpha), _number("beta", beta), _number("eps", eps), 0)
    if not a.eps > 0:  # (of the fp32 number)
        raise EntqError(EINVAL, f"eps is {eps!r}: a positive number is required")
    return index, a


def block(x, branch=None, out=None, post=None, gate=None, pre=None, y=None, y_scales=None,
          alpha=1.0, beta=1.0, eps=1e-6, stream=None):
    """The state into ``out`` (x's type [M, N], required with a branch; x
    itself is allowed) and its norm into ``y``: x's type [M, N], or int8 codes
    with ``y_scales`` (float32 [M]). Without a branch the state is x and only y
    is written. y None: no norm (pre is then None too)."""
    index, a = _describe(x, branch, post, gate, pre, alpha, beta, eps)
    shape, kind, n = x.shape, a.type, a.cols
    if (branch is None) != (out is None):
        raise EntqError(EINVAL, "out is required with a branch and takes nothing without one")
    if branch is None and y is None:
        raise EntqError(EINVAL, "neither a branch nor y: there is nothing to do")
    if (y is None) != (pre is None):
        raise EntqError(EINVAL, "y and pre go together")
    ldo, ldy, y_type, yp, sp, op = n, n, kind, 0, 0, 0
    if out is not None:
        ldo, op = _matrix("out", out, index, (kind,), shape)[1], out.data_ptr()
    if y is not None:
        y_type, ldy = _matrix("y", y, index, (kind, _I8), shape)
        yp = y.data_ptr()
    if (y_type == _I8) != (y_scales is not None):
        raise EntqError(EINVAL, "y_scales go with int8 codes in y")
    if y_scales is not None:
        sp = _vector("y_scales", y_scales, index, a.rows)
    _enqueue("entq_norm_block",
             lambda w, b, s: lib().entq_norm_block(a, op, ldo, yp, y_type, ldy, sp, s),
             0, index, stream, None)


def block_backward(state, dout=None, dy=None, branch=None, post=None, gate=None, pre=None,
                   dx=None, dbranch=None, dgate=None, dpre=None, dpost=None, alpha=1.0, beta=1.0,
                   eps=1e-6, stream=None, workspace=None):
    """Gradients of ``block`` for dout = dL/dstate and dy = dL/dy (the state's
    type, [M, N]; None: it has none, but one is required). state: what the
    forward call wrote to out (x without a branch); branch, post, gate, pre and
    the numbers as there. dx and dbranch: the state's type [M, N]; dgate: as
    the gate; dpre and dpost: float32 [N]. A gradient whose tensor is None is
    not computed."""
    index, a = _describe(state, branch, post, gate, pre, alpha, beta, eps, "state")
    shape, n = state.shape, a.cols
    if dout is None and dy is None:
        raise EntqError(EINVAL, "dout or dy is required")
    for name, t, need, why in (("dy", dy, pre, "pre"), ("dpre", dpre, dy, "dy"),
                               ("dbranch", dbranch, branch, "a branch"),
                               ("dpost", dpost, post, "post"), ("dgate", dgate, gate, "a gate")):
        if t is not None and need is None:
            raise EntqError(EINVAL, f"{name} without {why}")
    mats = []
    for name, t in (("dout", dout), ("dy", dy), ("dx", dx), ("dbranch", dbranch)):
        ld = n
        if t is not None:
            _, ld = _matrix(name, t, index, (a.type,), shape)
            if name in ("dout", "dy"):
                _no_graph(name, t)
        mats += [0 if t is None else t.data_ptr(), ld]
    ldg = n
    if dgate is not None:
        kind, ldg = _gate("dgate", dgate, a.type, index, *shape)
        if kind != a.gate_kind:
            raise EntqError(EINVAL, f"dgate has shape {tuple(dgate.shape)}, the gate "
                                    f"{tuple(gate.shape)}")
    gp = 0 if dgate is None else dgate.data_ptr()
    pp = 0 if dpre is None else _vector("dpre", dpre, index, n)
    qp = 0 if dpost is None else _vector("dpost", dpost, index, n)
    L = lib()
    _enqueue("entq_norm_block_backward",
             lambda p, b, s: L.entq_norm_block_backward(a, *mats, gp, ldg, pp, qp, p, b, s),
             L.entq_norm_block_backward_workspace_bytes(a), index, stream, workspace)


def workspace_bytes(state, branch=None, post=None, gate=None, pre=None):
    """Bytes of workspace that block_backward takes for these tensors."""
    _, a = _describe(state, branch, post, gate, pre, 1, 1, 1)
    return int(lib().entq_norm_block_backward_workspace_bytes(a))
