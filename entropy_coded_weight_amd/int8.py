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
"""
from __future__ import annotations

import ctypes

import torch

from . import EINVAL, EntqError, _check, lib

ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2, "relu": 3}
MAX_COLS = 131071  # keeps every sum of code products inside int32

_TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.int8: 3}
_BF16, _F16, _F32, _I8 = 0, 1, 2, 3


class _Rows(ctypes.Structure):  # entq_rows
    _fields_ = [("data", ctypes.c_void_p), ("ld", ctypes.c_uint64), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_uint32), ("cols", ctypes.c_uint32), ("type", ctypes.c_int32),
                ("reserved", ctypes.c_uint32)]


def _matrix(name, t, device, types, shape=None):
    """(type, row stride) of a 2-D device matrix with unit-stride rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise EntqError(EINVAL, f"{name}: a torch tensor on a GPU is required")
    if device is not None and t.device != device:
        raise EntqError(EINVAL, f"{name} is on {t.device}, expected {device}")
    kind = _TYPES.get(t.dtype)
    if kind not in types:
        raise EntqError(EINVAL, f"{name} has dtype {t.dtype}")
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise EntqError(EINVAL, f"{name} has shape {tuple(t.shape)}"
                                + ("" if shape is None else f", expected {tuple(shape)}"))
    ld, unit = t.stride()
    rows, cols = t.shape
    if rows <= 1 or cols == 0:
        ld = max(ld, cols)
    if (unit != 1 and cols > 1) or ld < cols:
        raise EntqError(EINVAL, f"{name}: strides {t.stride()}; rows of unit stride that do not "
                                "overlap are required")
    return kind, ld


def _vector(name, t, device, n):
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise EntqError(EINVAL, f"{name}: a torch tensor on {device} is required")
    if t.dtype != torch.float32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise EntqError(EINVAL, f"{name}: {t.dtype} {tuple(t.shape)}; a contiguous float32 vector "
                                f"of {n} is required")
    return t.data_ptr()


def _x_rows(x, x_scales, types=(_BF16, _F16, _F32, _I8)):
    kind, ld = _matrix("x", x, None, types)
    m, k = x.shape
    if k > MAX_COLS:
        raise EntqError(EINVAL, f"x has {k} columns, at most {MAX_COLS} are taken")
    if kind == _I8:
        s = _vector("x_scales", x_scales, x.device, m)
    elif x_scales is not None:
        raise EntqError(EINVAL, f"x_scales go with int8 codes, x has dtype {x.dtype}")
    else:
        s = 0
    return _Rows(x.data_ptr(), ld, s, m, k, kind, 0)


def _w_rows(name, w, scales, x, shape=None):
    _, ld = _matrix(name, w, x.device, (_I8,), shape)
    n, k = w.shape
    if k != x.shape[1]:
        raise EntqError(EINVAL, f"{name} has {k} columns, x has {x.shape[1]}")
    return _Rows(w.data_ptr(), ld, _vector(name + "_scales", scales, x.device, n), n, k, _I8, 0)


def _grad_rows(name, t, x, n):
    kind, ld = _matrix(name, t, x.device, (_BF16, _F16), (x.shape[0], n))
    return _Rows(t.data_ptr(), ld, 0, t.shape[0], n, kind, 0)


def _enqueue(what, call, need, device, stream, workspace):
    """Runs ``call(workspace pointer, bytes, stream handle)`` on ``stream``
    with a workspace of ``need`` bytes, allocated on that stream when none is
    given (so that its memory is ordered with what else uses it there)."""
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return _enqueue(what, call, need, device, stream, workspace)
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != device:
            raise EntqError(EINVAL, f"workspace: a torch tensor on {device} is required")
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise EntqError(EINVAL, "workspace: a contiguous uint8 tensor is required")
        if workspace.numel() < need:
            raise EntqError(EINVAL, f"workspace holds {workspace.numel()} bytes, {need} needed")
    if stream is None:
        stream = torch.cuda.current_stream(device)
    elif isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                  else torch.cuda.default_stream(device))
    if workspace is None and need:
        if stream == torch.cuda.current_stream(device):
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(need, dtype=torch.uint8, device=device)
    ptr, n = (workspace.data_ptr(), workspace.numel()) if workspace is not None else (0, 0)
    _check(call(ptr, n, stream.cuda_stream), what)


def quantize_rows(x, codes, scales, stream=None):
    """Codes and scales of the rows of x (bfloat16, float16 or float32
    [M, K]) into ``codes`` (int8 [M, K]) and ``scales`` (float32 [M]):
    scale = max(|x|) / 127 (at least 2^-100), code = x / scale rounded half
    to even. A row with a NaN or an infinity gets a NaN scale and codes 0."""
    kind, ld = _matrix("x", x, None, (_BF16, _F16, _F32))
    m, k = x.shape
    if k > MAX_COLS:
        raise EntqError(EINVAL, f"x has {k} columns, at most {MAX_COLS} are taken")
    _, ldc = _matrix("codes", codes, x.device, (_I8,), x.shape)
    s = _vector("scales", scales, x.device, m)
    r = _Rows(x.data_ptr(), ld, 0, m, k, kind, 0)
    _enqueue("entq_quantize_rows",
             lambda w, n, st: lib().entq_quantize_rows(ctypes.byref(r), codes.data_ptr(), ldc, s, st),
             0, x.device, stream, None)


def gemm(x, x_scales, w, w_scales, y, stream=None, workspace=None):
    """Y = X . W^T into y (bfloat16, float16 or float32 [M, N]):
    y[m][n] = sx[m] sw[n] sum_k x[m][k] w[n][k], the sum exact in int32."""
    xr = _x_rows(x, x_scales)
    wr = _w_rows("w", w, w_scales, x)
    kind, ldy = _matrix("y", y, x.device, (_BF16, _F16, _F32), (x.shape[0], w.shape[0]))
    L = lib()
    a, b = ctypes.byref(xr), ctypes.byref(wr)
    _enqueue("entq_int8_gemm",
             lambda p, n, s: L.entq_int8_gemm(a, b, y.data_ptr(), kind, ldy, p, n, s),
             L.entq_int8_gemm_workspace_bytes(a, b), x.device, stream, workspace)


def gated(x, x_scales, gate, gate_scales, up, up_scales, h, activation="silu", stream=None,
          workspace=None):
    """H = act(X . gate^T) * (X . up^T) into h (bfloat16, float16 or float32
    [M, N]), both products, the activation and the product in one kernel.
    activation: "silu", "gelu", "gelu_tanh" or "relu"."""
    xr = _x_rows(x, x_scales)
    gr = _w_rows("gate", gate, gate_scales, x)
    ur = _w_rows("up", up, up_scales, x, gate.shape)
    kind, ldh = _matrix("h", h, x.device, (_BF16, _F16, _F32), (x.shape[0], gate.shape[0]))
    act = _activation(activation)
    L = lib()
    a, g, u = ctypes.byref(xr), ctypes.byref(gr), ctypes.byref(ur)
    _enqueue("entq_int8_gated",
             lambda p, n, s: L.entq_int8_gated(a, g, u, act, h.data_ptr(), kind, ldh, p, n, s),
             L.entq_int8_gated_workspace_bytes(a, g, u), x.device, stream, workspace)


def gemm_backward(dy, x, x_scales, w, w_scales, dx=None, dw_scales=None, stream=None,
                  workspace=None):
    """Gradients of ``gemm`` for dy (bfloat16 or float16 [M, N]): dx (dy's
    type, [M, K]; the quantiser of x passed straight through) and dw_scales
    (float32 [N]). x: the int8 codes of the forward pass. A gradient whose
    tensor is None is not computed."""
    xr = _x_rows(x, x_scales, (_I8,))
    wr = _w_rows("w", w, w_scales, x)
    dr = _grad_rows("dy", dy, x, w.shape[0])
    dxp, lddx = _dx(dx, dy, x)
    ds = _vector("dw_scales", dw_scales, x.device, w.shape[0]) if dw_scales is not None else 0
    L = lib()
    d, a, b = ctypes.byref(dr), ctypes.byref(xr), ctypes.byref(wr)
    _enqueue("entq_int8_gemm_backward",
             lambda p, n, s: L.entq_int8_gemm_backward(d, a, b, dxp, lddx, ds, p, n, s),
             L.entq_int8_gemm_backward_workspace_bytes(d, a, b), x.device, stream, workspace)


def gated_backward(dh, x, x_scales, gate, gate_scales, up, up_scales, dx=None,
                   dgate_scales=None, dup_scales=None, activation="silu", stream=None,
                   workspace=None):
    """Gradients of ``gated`` for dh (bfloat16 or float16 [M, N]): dx (dh's
    type, [M, K]), dgate_scales and dup_scales (float32 [N]); x, None and the
    rest as ``gemm_backward``."""
    xr = _x_rows(x, x_scales, (_I8,))
    gr = _w_rows("gate", gate, gate_scales, x)
    ur = _w_rows("up", up, up_scales, x, gate.shape)
    n = gate.shape[0]
    dr = _grad_rows("dh", dh, x, n)
    dxp, lddx = _dx(dx, dh, x)
    dsg = _vector("dgate_scales", dgate_scales, x.device, n) if dgate_scales is not None else 0
    dsu = _vector("dup_scales", dup_scales, x.device, n) if dup_scales is not None else 0
    act = _activation(activation)
    L = lib()
    d, a, g, u = ctypes.byref(dr), ctypes.byref(xr), ctypes.byref(gr), ctypes.byref(ur)
    _enqueue("entq_int8_gated_backward",
             lambda p, b, s: L.entq_int8_gated_backward(d, a, g, u, act, dxp, lddx, dsg, dsu, p, b, s),
             L.entq_int8_gated_backward_workspace_bytes(d, a, g, u), x.device, stream, workspace)


def _activation(name):
    act = ACTIVATIONS.get(name)
    if act is None:
        raise EntqError(EINVAL, f"activation {name!r}: one of {', '.join(ACTIVATIONS)}")
    return act


def _dx(dx, dy, x):
    if dx is None:
        return 0, x.shape[1]
    _, ld = _matrix("dx", dx, x.device, (_TYPES[dy.dtype],), x.shape)
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
    args = [_x_rows(x, x_scales)]
    for i in range(0, len(weights_and_scales), 2):
        args.append(_w_rows(f"w{i // 2}", *weights_and_scales[i:i + 2], x))
    if op.endswith("backward"):
        args.insert(0, _grad_rows("dy", dy, x, weights_and_scales[0].shape[0]))
    return int(getattr(lib(), f"entq_int8_{op}_workspace_bytes")(*map(ctypes.byref, args)))
