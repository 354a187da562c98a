"""A mixture-of-experts layer on compressed Int8 weights, for the few tokens of
a decode step (the entq_moe_few call of include/entq.h). For tokens x [M, D]:

    l = x . router^T, the top_k experts of largest l chosen,
    p = softmax of l over the chosen (normalize) or over all experts,
    y = sum over the chosen of p_e ((act(x . gate_e^T) * (x . up_e^T)) . down_e^T)

with every expert's products those of ``int8.gated`` and ``int8.gemm``: x and
the hidden values are quantised to int8 per row. Only the codes of the chosen
experts are read. ``MixtureOfExperts`` is the layer on a plan: the experts are
decoded to codes, then used for any number of steps. Streams, workspaces, and
what needs an autograd graph are as in ``int8``; there is no backward pass.
"""
from __future__ import annotations

import torch

from . import EINVAL, KIND_INT8, EntqError, Experts, Plan, Rows, lib
from .feed_forward import DecodedCodes
from .int8 import (_BF16, _F16, _F32, MAX_COLS, _activation, _check_activations, _enqueue, _gpu,
                   _matrix, _no_graph)

MAX_TOKENS = 64
MAX_EXPERTS = 256
MAX_TOP = 32

_FLOATS = (_BF16, _F16, _F32)


def _codes3(name, t, index, shape):
    """(address, row stride, expert stride) of int8 codes [E, rows, cols]."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise EntqError(EINVAL, f"{name}: a torch tensor on cuda:{index} is required")
    if t.dtype != torch.int8 or t.dim() != 3 or any(s is not None and s != n
                                                    for s, n in zip(shape, t.shape)):
        raise EntqError(EINVAL, f"{name}: {t.dtype} {tuple(t.shape)}; int8 "
                                f"[{', '.join('any' if s is None else str(s) for s in shape)}] is "
                                "required")
    e, rows, cols = t.shape
    if min(e, rows, cols) < 1:
        raise EntqError(EINVAL, f"{name} has shape {tuple(t.shape)}")
    stride, ld, unit = t.stride()
    ld = ld if rows > 1 else max(ld, cols)
    stride = stride if e > 1 else rows * ld
    if (unit != 1 and cols > 1) or ld < cols or stride < (rows - 1) * ld + cols:
        raise EntqError(EINVAL, f"{name}: strides {t.stride()}; rows of unit stride and experts "
                                "that do not overlap are required")
    return t.data_ptr(), ld, stride


def _scales2(name, t, index, shape):
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise EntqError(EINVAL, f"{name}: a torch tensor on cuda:{index} is required")
    if t.dtype != torch.float32 or t.shape != shape:
        raise EntqError(EINVAL, f"{name}: {t.dtype} {tuple(t.shape)}; float32 {tuple(shape)} is "
                                "required")
    stride = t.stride(0) if shape[0] > 1 else shape[1]
    if (t.stride(1) != 1 and shape[1] > 1) or stride < shape[1]:
        raise EntqError(EINVAL, f"{name}: strides {t.stride()}; a unit stride along each expert's "
                                "scales is required")
    return t.data_ptr(), stride


def _describe(x, router, gate, gate_scales, up, up_scales, down, down_scales, top_k, activation,
              normalize):
    index = _gpu("x", x)
    kind, ldx = _matrix("x", x, index, _FLOATS)
    _no_graph("x", x)
    m, d = x.shape
    if m > MAX_TOKENS:
        raise EntqError(EINVAL, f"{m} tokens, at most {MAX_TOKENS} are taken")
    gp = _codes3("gate", gate, index, (None, None, d))
    e, f, _ = gate.shape
    up_ = _codes3("up", up, index, (e, f, d))
    dn = _codes3("down", down, index, (e, None, f))
    n = down.shape[1]
    if e > MAX_EXPERTS or max(d, f) > MAX_COLS or n > 1 << 22:
        raise EntqError(EINVAL, f"{e} experts of {d} x {f} x {n}: at most {MAX_EXPERTS} experts, "
                                f"{MAX_COLS} columns and {1 << 22} results are taken")
    if not isinstance(top_k, int) or not 1 <= top_k <= min(e, MAX_TOP):
        raise EntqError(EINVAL, f"top_k {top_k!r}: 1 to {min(e, MAX_TOP)} of {e} experts are taken")
    rkind, ldr = _matrix("router", router, index, _FLOATS, (e, d))
    _no_graph("router", router)
    a = Experts(e, top_k, f, n, _activation(activation), 1 if normalize else 0, rkind, 0,
                router.data_ptr(), ldr)
    scales = (_scales2("gate_scales", gate_scales, index, (e, f)),
              _scales2("up_scales", up_scales, index, (e, f)),
              _scales2("down_scales", down_scales, index, (e, n)))
    for i, (w, s) in enumerate(zip((gp, up_, dn), scales)):
        a.weights[i], a.ld[i], a.stride[i] = w
        a.scales[i], a.scale_stride[i] = s
    return index, Rows(x.data_ptr(), ldx, 0, m, d, kind, 0), a


def _choice(name, t, dtype, index, shape):
    if t is None:
        return 0
    if not isinstance(t, torch.Tensor) or t.get_device() != index or t.dtype != dtype or \
            t.shape != shape or not t.is_contiguous():
        raise EntqError(EINVAL, f"{name}: a contiguous {dtype} tensor {tuple(shape)} on "
                                f"cuda:{index} is required")
    return t.data_ptr()


def few(x, router, gate, gate_scales, up, up_scales, down, down_scales, y, top_k,
        activation="silu", normalize=True, experts=None, weights=None, stream=None,
        workspace=None):
    """The layer for x (bfloat16, float16 or float32 [M, D], M up to
    MAX_TOKENS) into y (any of these types [M, N]). router: any of these types
    [E, D]; gate and up: int8 codes [E, F, D] with float32 scales [E, F]; down:
    [E, N, F] with [E, N]; unit stride along the last dimension, any other
    strides and alignment. experts (int32 [M, top_k]) and weights (float32 [M,
    top_k]), unless None: the chosen experts by descending l (equal ones: the
    lowest index first) and their p."""
    index, a, e = _describe(x, router, gate, gate_scales, up, up_scales, down, down_scales, top_k,
                            activation, normalize)
    kind, ldy = _matrix("y", y, index, _FLOATS, (a.rows, e.out))
    chosen = (a.rows, top_k)
    ep = _choice("experts", experts, torch.int32, index, chosen)
    wp = _choice("weights", weights, torch.float32, index, chosen)
    L = lib()
    _enqueue("entq_moe_few",
             lambda p, n, s: L.entq_moe_few(a, e, y.data_ptr(), kind, ldy, ep, wp, p, n, s),
             L.entq_moe_few_workspace_bytes(a, e), index, stream, workspace)


def workspace_bytes(x, router, gate, gate_scales, up, up_scales, down, down_scales, top_k):
    """Bytes of workspace that ``few`` takes for these tensors."""
    _, a, e = _describe(x, router, gate, gate_scales, up, up_scales, down, down_scales, top_k,
                        "silu", True)
    return int(lib().entq_moe_few_workspace_bytes(a, e))


class MixtureOfExperts(DecodedCodes):
    """p: a plan of Int8 tensors, for each expert gate [F, D], up [F, D] and
    down [N, F], the experts one after the other (equal steps upwards between
    their codes and between their scales, of which each expert has its own);
    scales: device float32 with the plan's row scales; router: bfloat16,
    float16 or float32 [E, D]. ``decode`` fills the code buffer (``codes``:
    device int8, at least out_elems; None: the layer's own), which ``forward``
    then uses. Streams and the buffer are as in ``feed_forward.FeedForward``."""

    def __init__(self, p: Plan, scales, router, top_k, activation="silu", normalize=True,
                 codes=None):
        t = p.tensors
        n = p.n_tensors // 3
        if not n or p.n_tensors % 3 or any(int(k) & 0xFF != KIND_INT8 for k in t["kind"]):
            raise EntqError(EINVAL, "a mixture of experts is three Int8 tensors for each expert: "
                                    "gate, up, down")
        shapes = [(int(r["rows"]), int(r["cols"])) for r in t]
        (f, d), (_, _), (out, f2) = shapes[:3]
        if shapes != [(f, d), (f, d), (out, f)] * n or f2 != f:
            raise EntqError(EINVAL, f"tensors of shapes {sorted(set(shapes))}: gate and up of one "
                                    "shape, down a column for each of their rows, every expert "
                                    "alike")
        at = [[int(v) for v in t[key]] for key in ("out_elem_offset", "scale_row_offset")]
        steps = [a[3] - a[0] if n > 1 else 0 for a in at]
        if any(a[i] != a[i % 3] + i // 3 * s for a, s in zip(at, steps) for i in range(3 * n)):
            raise EntqError(EINVAL, "the experts' tensors do not lie at equal steps")
        if n > 1 and min(steps) <= 0:
            raise EntqError(EINVAL, "the experts' tensors lie backwards or share their scales: each "
                                    "expert is to have its own, after those of the one before")
        super().__init__(p, scales, codes)
        flat, rows = self.codes.view(-1), self.scales.view(-1)
        self._w = []
        for i, (r, c) in enumerate(shapes[:3]):
            self._w += [flat.as_strided((n, r, c), (steps[0] if n > 1 else r * c, c, 1),
                                        flat.storage_offset() + at[0][i]),
                        rows.as_strided((n, r), (steps[1] if n > 1 else r, 1),
                                        rows.storage_offset() + at[1][i])]
        self.router, self.top_k = router, top_k
        self.activation, self.normalize = activation, normalize
        self.experts, self.width, self.hidden, self.out = n, d, f, out
        # (every check of the call, before the first token comes)
        _describe(torch.empty(0, d, device=p.device), router, *self._w, top_k, activation, normalize)

    def forward(self, x, y, experts=None, weights=None, stream=None):
        """y = layer(x): x bfloat16, float16 or float32 [m, D], y of any of
        these types [m, N]; experts and weights as in ``few``. Tokens beyond
        MAX_TOKENS run in groups of that many, each of which reads its experts'
        codes again."""
        index = self.plan.device.index
        m = _check_activations("x", x, index, self.width)
        _matrix("y", y, index, _FLOATS, (m, self.out))
        _choice("experts", experts, torch.int32, index, (m, self.top_k))
        _choice("weights", weights, torch.float32, index, (m, self.top_k))
        part = lambda t, r: None if t is None else t[r:r + MAX_TOKENS]  # noqa: E731
        with self._using_codes(stream):
            for r in range(0, m, MAX_TOKENS):
                few(part(x, r), self.router, *self._w, part(y, r), self.top_k, self.activation,
                    self.normalize, part(experts, r), part(weights, r))
