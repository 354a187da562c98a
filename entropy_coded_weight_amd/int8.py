"""Products on int8 weight codes: quantised activations times the Int8 codes
that ``decode(..., OUT_CODES)`` leaves in device memory, the gated
feed-forward kernel on such codes, and the backward pass of both (the
entq_int8_* calls and entq_quantize_rows of include/entq.h).

Weights are int8 [N, K] codes (unit stride along K, any row stride and
alignment) with float32 scales [N]; activations are either bfloat16, float16
or float32 [M, K] tensors with ``x_scales=None`` (quantised inside the call)
or int8 codes with float32 scales [M], as ``quantize_rows`` writes them.
Results go to tensors of the caller. ``stream`` is a torch stream, a raw
stream handle or None for the current stream; ``workspace`` a device uint8
tensor of at least ``workspace_bytes(...)`` bytes, or None to allocate one
for the call.

The calls record no autograd graph. Activations and incoming gradients that
require a gradient are refused while gradients are enabled, since the graph
would end there unnoticed: a torch.autograd.Function around the forward and
the backward call connects them (inside it gradients are disabled). Scales may
be parameters; their gradients are what the backward calls write.
"""
from __future__ import annotations

import torch

from . import EINVAL, EntqError, Rows, _check, lib

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
MAX_COLS = 131071  # keeps every sum of code products inside int32

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int8: 3}
_BF16, _F16, _F32, _I8 = 0, 1, 2, 3


def _matrix(name, t, index, types, shape=None):
    """(type, row stride) of a 2-D matrix with unit-stride rows on GPU
    ``index``."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise EntqError(EINVAL, f"{name}: a torch tensor on a GPU is required")
    if t.get_device() != index:
        raise EntqError(EINVAL, f"{name} is on {t.device}, expected cuda:{index}")
    kind = _TYPES.get(t.dtype)
    if kind not in types:
        raise EntqError(EINVAL, f"{name} has dtype {t.dtype}")
    size = t.shape
    if len(size) != 2 or (shape is not None and size != shape):
        raise EntqError(EINVAL, f"{name} has shape {tuple(size)}"
                                + ("" if shape is None else f", expected {tuple(shape)}"))
    ld, unit = t.stride()
    rows, cols = size
    if unit != 1 or ld < cols:
        if rows <= 1 or cols == 0:
            ld = max(ld, cols)
        if (unit != 1 and cols > 1) or ld < cols:
            raise EntqError(EINVAL, f"{name}: strides {t.stride()}; rows of unit stride that do "
                                    "not overlap are required")
    return kind, ld


def _no_graph(name, t):
    if t.requires_grad and torch.is_grad_enabled():
        raise EntqError(EINVAL, f"{name} requires a gradient, which this call does not record: call "
                                "it from a torch.autograd.Function, under torch.no_grad() or "
                                f"with {name}.detach()")


def _vector(name, t, index, n):
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise EntqError(EINVAL, f"{name}: a torch tensor on cuda:{index} is required")
    if t.dtype != torch.float32 or t.shape != (n,) or not t.is_contiguous():
        raise EntqError(EINVAL, f"{name}: {t.dtype} {tuple(t.shape)}; a contiguous float32 vector "
                                f"of {n} is required")
    return t.data_ptr()


def _gpu(name, t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise EntqError(EINVAL, f"{name}: a torch tensor on a GPU is required")
    return t.get_device()


def _x_rows(x, x_scales, index, types=(_BF16, _F16, _F32, _I8)):
    kind, ld = _matrix("x", x, index, types)
    _no_graph("x", x)
    m, k = x.shape
    if k > MAX_COLS:
        raise EntqError(EINVAL, f"x has {k} columns, at most {MAX_COLS} are taken")
    if kind == _I8:
        s = _vector("x_scales", x_scales, index, m)
    elif x_scales is not None:
        raise EntqError(EINVAL, f"x_scales go with int8 codes, x has dtype {x.dtype}")
    else:
        s = 0
    return Rows(x.data_ptr(), ld, s, m, k, kind, 0)


def _check_activations(name, x, index, columns, types=(_BF16, _F16, _F32)):
    """Activations of one of ``types`` for weights of that many columns: what a
    call that runs several products checks before the first. Returns their
    number of tokens."""
    _matrix(name, x, index, types)
    _no_graph(name, x)
    if x.shape[1] != columns:
        raise EntqError(EINVAL, f"{name} has {x.shape[1]} columns, the weights have {columns}")
    if columns > MAX_COLS:
        raise EntqError(EINVAL, f"{name} has {columns} columns, at most {MAX_COLS} are taken")
    return x.shape[0]


def _check_result(name, y, index, rows, n):
    _matrix(name, y, index, (_BF16, _F16, _F32), (rows, n))


def _w_rows(name, w, scales, index, columns, shape=None):
    _, ld = _matrix(name, w, index, (_I8,), shape)
    n, k = w.shape
    if k != columns:
        raise EntqError(EINVAL, f"{name} has {k} columns, x has {columns}")
    return Rows(w.data_ptr(), ld, _vector(name + "_scales", scales, index, n), n, k, _I8, 0)


def _grad_rows(name, t, index, rows, n):
    kind, ld = _matrix(name, t, index, (_BF16, _F16), (rows, n))
    _no_graph(name, t)
    return Rows(t.data_ptr(), ld, 0, rows, n, kind, 0)


def _enqueue(what, call, need, index, stream, workspace):
    """Runs ``call(workspace pointer, bytes, stream handle)`` on ``stream``
    with a workspace of ``need`` bytes, allocated on that stream when none is
    given (so that its memory is ordered with what else uses it there)."""
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _enqueue(what, call, need, index, stream, workspace)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.get_device() != index:
            raise EntqError(EINVAL, f"workspace: a torch tensor on cuda:{index} is required")
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise EntqError(EINVAL, "workspace: a contiguous uint8 tensor is required")
        if workspace.numel() < need:
            raise EntqError(EINVAL, f"workspace holds {workspace.numel()} bytes, {need} needed")
    if stream is None:
        handle = _current_stream(index)
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=index)
    else:
        if isinstance(stream, int):
            stream = (torch.cuda.ExternalStream(stream, device=index) if stream
                      else torch.cuda.default_stream(index))
        handle = stream.cuda_stream
        if workspace is None and need:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=index)
    if workspace is None:
        _check(call(0, 0, handle), what)
    else:
        _check(call(workspace.data_ptr(), workspace.numel(), handle), what)


def _current_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


# the same handle without a Stream object around it (1.9 us of a call's 10)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def quantize_rows(x, codes, scales, stream=None):
    """Codes and scales of the rows of x (bfloat16, float16 or float32
    [M, K]) into ``codes`` (int8 [M, K]) and ``scales`` (float32 [M]):
    scale = max(|x|) / 127 (at least 2^-100), code = x / scale rounded half
    to even. A row with a NaN or an infinity gets a NaN scale and codes 0."""
    index = _gpu("x", x)
    r = _x_rows(x, None, index, (_BF16, _F16, _F32))
    _, ldc = _matrix("codes", codes, index, (_I8,), x.shape)
    s = _vector("scales", scales, index, r.rows)
    _enqueue("entq_quantize_rows",
             lambda w, n, st: lib().entq_quantize_rows(r, codes.data_ptr(), ldc, s, st),
             0, index, stream, None)


def gemm(x, x_scales, w, w_scales, y, stream=None, workspace=None):
    """Y = X . W^T into y (bfloat16, float16 or float32 [M, N]):
    y[m][n] = sx[m] sw[n] sum_k x[m][k] w[n][k], the sum exact in int32."""
    index = _gpu("x", x)
    a = _x_rows(x, x_scales, index)
    b = _w_rows("w", w, w_scales, index, a.cols)
    kind, ldy = _matrix("y", y, index, (_BF16, _F16, _F32), (a.rows, b.rows))
    L = lib()
    _enqueue("entq_int8_gemm",
             lambda p, n, s: L.entq_int8_gemm(a, b, y.data_ptr(), kind, ldy, p, n, s),
             L.entq_int8_gemm_workspace_bytes(a, b), index, stream, workspace)


def gated(x, x_scales, gate, gate_scales, up, up_scales, h, activation="silu", stream=None,
          workspace=None):
    """H = act(X . gate^T) * (X . up^T) into h (bfloat16, float16 or float32
    [M, N]), both products, the activation and the product in one kernel.
    activation: "silu", "gelu", "gelu_tanh" or "relu"."""
    index = _gpu("x", x)
    a = _x_rows(x, x_scales, index)
    g = _w_rows("gate", gate, gate_scales, index, a.cols)
    u = _w_rows("up", up, up_scales, index, a.cols, gate.shape)
    kind, ldh = _matrix("h", h, index, (_BF16, _F16, _F32), (a.rows, g.rows))
    act = _activation(activation)
    L = lib()
    _enqueue("entq_int8_gated",
             lambda p, n, s: L.entq_int8_gated(a, g, u, act, h.data_ptr(), kind, ldh, p, n, s),
             L.entq_int8_gated_workspace_bytes(a, g, u), index, stream, workspace)


def gemm_backward(dy, x, x_scales, w, w_scales, dx=None, dw_scales=None, stream=None,
                  workspace=None):
    """Gradients of ``gemm`` for dy (bfloat16 or float16 [M, N]): dx (dy's
    type, [M, K]; the quantiser of x passed straight through) and dw_scales
    (float32 [N]). x: the int8 codes of the forward pass. A gradient whose
    tensor is None is not computed."""
    index = _gpu("x", x)
    a = _x_rows(x, x_scales, index, (_I8,))
    b = _w_rows("w", w, w_scales, index, a.cols)
    d = _grad_rows("dy", dy, index, a.rows, b.rows)
    dxp, lddx = _dx(dx, d, x, index)
    ds = _vector("dw_scales", dw_scales, index, b.rows) if dw_scales is not None else 0
    L = lib()
    _enqueue("entq_int8_gemm_backward",
             lambda p, n, s: L.entq_int8_gemm_backward(d, a, b, dxp, lddx, ds, p, n, s),
             L.entq_int8_gemm_backward_workspace_bytes(d, a, b), index, stream, workspace)


def gated_backward(dh, x, x_scales, gate, gate_scales, up, up_scales, dx=None,
                   dgate_scales=None, dup_scales=None, activation="silu", stream=None,
                   workspace=None):
    """Gradients of ``gated`` for dh (bfloat16 or float16 [M, N]): dx (dh's
    type, [M, K]), dgate_scales and dup_scales (float32 [N]); x, None and the
    rest as ``gemm_backward``."""
    index = _gpu("x", x)
    a = _x_rows(x, x_scales, index, (_I8,))
    g = _w_rows("gate", gate, gate_scales, index, a.cols)
    u = _w_rows("up", up, up_scales, index, a.cols, gate.shape)
    d = _grad_rows("dh", dh, index, a.rows, g.rows)
    dxp, lddx = _dx(dx, d, x, index)
    dsg = _vector("dgate_scales", dgate_scales, index, g.rows) if dgate_scales is not None else 0
    dsu = _vector("dup_scales", dup_scales, index, g.rows) if dup_scales is not None else 0
    act = _activation(activation)
    L = lib()
    _enqueue("entq_int8_gated_backward",
             lambda p, n, s: L.entq_int8_gated_backward(d, a, g, u, act, dxp, lddx, dsg, dsu, p, n, s),
             L.entq_int8_gated_backward_workspace_bytes(d, a, g, u), index, stream, workspace)


def _activation(name):
    act = ACTIVATIONS.get(name)
    if act is None:
        raise EntqError(EINVAL, f"activation {name!r}: one of {', '.join(ACTIVATIONS)}")
    return act


def _dx(dx, d, x, index):
    if dx is None:
        return 0, x.shape[1]
    _, ld = _matrix("dx", dx, index, (d.type,), x.shape)
    return dx.data_ptr(), ld


def workspace_bytes(op, x, x_scales, *weights_and_scales, dy=None):
    """Bytes of workspace a call takes: op "gemm", "gated", "gemm_backward"
    or "gated_backward", then x, x_scales and the weights and scales as the
    call takes them (and dy, the incoming gradient, for a backward call)."""
    two = op.startswith("gated")
    if op not in ("gemm", "gated", "gemm_backward", "gated_backward") or \
            len(weights_and_scales) != (4 if two else 2):
        raise EntqError(EINVAL, f"workspace_bytes of {op!r} with {len(weights_and_scales)} "
                                "weights and scales")
    index = _gpu("x", x)
    args = [_x_rows(x, x_scales, index)]
    for i in range(0, len(weights_and_scales), 2):
        args.append(_w_rows(f"w{i // 2}", *weights_and_scales[i:i + 2], index, args[0].cols))
    if op.endswith("backward"):
        args.insert(0, _grad_rows("dy", dy, index, args[0].rows, args[1].rows))
    return int(getattr(lib(), f"entq_int8_{op}_workspace_bytes")(*args))
