"""Products of compressed weights with activations for any number of rows.

Up to FUSED_MAX_ROWS activation rows (the decode phase of inference) the
product is the fused decode + product (decode_gemm_tiles for tensors in tile
order, else decode_gemm): the bf16 weights are never written. With
more rows (prefill) the product, not the decode, dominates a layer's time, so
the layer is decoded once to bf16 and each projection is one library GEMM --
weights expanded right before the block that uses them [EntQuant,
"Float8@2bits ...", technical summary §2 "Decodificación en Tiempo de
Inferencia"].
"""
from __future__ import annotations

import numpy as np

from . import (EINVAL, KIND_BF16EXP, KIND_INT8, LAYOUT_TILES, OUT_BF16, OUT_CODES, EntqError, Plan,
               _device_buffer, _gemm_io, decode, decode_gemm, decode_gemm_tiles)

FUSED_MAX_ROWS = 64


def linear(p: Plan, compressed, scales, xs, ys, weights=None, chunk_status=None, stream=None,
           workspace=None):
    """Y_t = X_t . W_t^T for every tensor t of the plan (xs[t]: device
    bfloat16 [m, >= cols]; ys[t]: device float32 [m, >= rows]; the same m for
    all). m <= FUSED_MAX_ROWS: decode_gemm_tiles when the plan's tensors are
    in tile order, else decode_gemm (workspace as there). More rows:
    the bf16 decode into `weights` (a device tensor of 2-byte elements, at
    least out_elems; allocated when None), then per tensor one library GEMM
    of the bf16 operands with fp32 accumulation and fp32 results, all on
    `stream` (a torch stream, a raw stream handle, or None for the current
    stream)."""
    import torch
    _gemm_io(p, xs, ys)  # shapes, dtypes and devices, as for the fused call
    m = xs[0].shape[0] if xs else 0
    tiles = bool(np.any(p.tensors["kind"] & LAYOUT_TILES))
    if m <= FUSED_MAX_ROWS:
        fused = decode_gemm_tiles if tiles else decode_gemm
        fused(p, compressed, scales, xs, ys, chunk_status, stream, workspace)
        return
    if p.adaptive:
        raise EntqError(EINVAL, "linear takes plans with per-tensor tables")
    if np.any((p.tensors["kind"] & 0xFF) == KIND_BF16EXP):
        raise EntqError(EINVAL, "linear takes Int8 and E4M3 tensors; exponent streams use "
                                "decode_gemm_bf16_split")
    own = weights is None
    if own:
        weights = torch.empty(p.out_elems, dtype=torch.int16, device=p.device)
    decode(p, compressed, weights, OUT_BF16, scales, chunk_status, stream)
    w = weights.view(torch.bfloat16)
    if stream is None:
        s = torch.cuda.current_stream(p.device)
    elif isinstance(stream, int):  # a raw stream handle, 0 for the null stream
        s = (torch.cuda.ExternalStream(stream, device=p.device) if stream
             else torch.cuda.default_stream(p.device))
    else:
        s = stream
    if own:
        weights.record_stream(s)  # allocated here, used on s
    with torch.cuda.stream(s):
        for t in range(p.n_tensors):
            rows, cols = int(p.tensors[t]["rows"]), int(p.tensors[t]["cols"])
            if rows * cols == 0:
                continue
            off = int(p.tensors[t]["out_elem_offset"])
            wt = w[off:off + rows * cols].view(rows, cols)
            ys[t][:, :rows].copy_(torch.mm(xs[t][:, :cols], wt.t(), out_dtype=torch.float32))


def linear_int8(p: Plan, compressed, scales, xs, ys, codes=None, chunk_status=None, stream=None):
    """Y_t = X_t . W_t^T for every tensor t of a plan of Int8 tensors, with the
    activations quantised to int8 per row: the plan is decoded to codes (half
    the bytes of bf16 weights) into ``codes`` (device int8, at least out_elems;
    allocated when None), then each product runs on the int8 matrix cores
    (int8.gemm). xs[t]: device bfloat16, float16 or float32 [m, cols]; ys[t]: any
    of these types [m, rows]; stream as in ``linear``."""
    import torch

    from . import int8
    from .feed_forward import _on
    if len(xs) != p.n_tensors or len(ys) != p.n_tensors:
        raise EntqError(EINVAL, f"{len(xs)} activation and {len(ys)} result matrices for "
                                f"{p.n_tensors} tensors")
    if np.any((p.tensors["kind"] & 0xFF) != KIND_INT8):
        raise EntqError(EINVAL, "linear_int8 takes Int8 tensors")
    _device_buffer(p, "scales", scales, p.scale_rows, dtypes=(torch.float32,))
    if codes is not None:
        _device_buffer(p, "codes", codes, p.out_elems, dtypes=(torch.int8,))
    for t, r in enumerate(p.tensors):
        m = int8._check_activations(f"x[{t}]", xs[t], p.device.index, int(r["cols"]))
        int8._check_result(f"y[{t}]", ys[t], p.device.index, m, int(r["rows"]))
    with _on(stream, p.device):
        if codes is None:
            codes = torch.empty(p.out_elems, dtype=torch.int8, device=p.device)
        decode(p, compressed, codes, OUT_CODES, None, chunk_status)
        codes, scales = codes.view(-1), scales.view(-1)
        for t, r in enumerate(p.tensors):
            rows, cols = int(r["rows"]), int(r["cols"])
            o, s = int(r["out_elem_offset"]), int(r["scale_row_offset"])
            int8.gemm(xs[t], None, codes[o:o + rows * cols].view(rows, cols), scales[s:s + rows], ys[t])


def distill_int8(p: Plan, compressed, scales, x, index, teacher, loss, dx=None, dscales=None,
                 dloss=None, teacher_lse=None, weight=None, temperature=1.0, codes=None,
                 tokens=1024, chunk_status=None, stream=None):
    """The distillation loss of a compressed output projection and its
    gradients, for any number of tokens: the plan's one Int8 tensor W [V, D]
    is decoded to codes; then, ``tokens`` tokens at a time, the fp32 logits
    x . W^T (int8.gemm), the losses with the logits' gradient in x's type
    (distill.loss_backward), and the gradients of x and of the row scales
    (int8.gemm_backward). The logits of all tokens are never in memory.

    x: device bfloat16 or float16 [m, D]; loss: float32 [m]; dx: x's type [m, D];
    dscales: float32 [V], the sum over all tokens in fp32; None: not computed
    (both None: the losses alone). index, teacher, dloss, teacher_lse, weight and
    temperature as in ``distill.loss_backward`` (a float16 gradient below 6e-8
    is 0, which a larger dloss mends); codes and stream as in ``linear_int8``."""
    import torch

    from . import distill, int8
    from .feed_forward import _on
    if p.n_tensors != 1 or (int(p.tensors[0]["kind"]) & 0xFF) != KIND_INT8:
        raise EntqError(EINVAL, "distill_int8 takes a plan of one Int8 tensor")
    v, d = int(p.tensors[0]["rows"]), int(p.tensors[0]["cols"])
    _device_buffer(p, "scales", scales, p.scale_rows, dtypes=(torch.float32,))
    if codes is not None:
        _device_buffer(p, "codes", codes, p.out_elems, dtypes=(torch.int8,))
    if not isinstance(tokens, int) or tokens < 1:
        raise EntqError(EINVAL, f"tokens is {tokens!r}: a positive number is required")
    at = p.device.index
    m = int8._check_activations("x", x, at, d, (int8._BF16, int8._F16))
    distill._entries(at, m, v, int8._F32, 0, v, index, teacher, teacher_lse, weight, temperature)
    int8._vector("loss", loss, at, m)
    if dloss is not None:
        int8._vector("dloss", dloss, at, m)
    if dx is not None:
        int8._matrix("dx", dx, at, (int8._TYPES[x.dtype],), x.shape)
    if dscales is not None:
        _device_buffer(p, "dscales", dscales, p.scale_rows, dtypes=(torch.float32,))
    with _on(stream, p.device):
        new = lambda *s, t=torch.float32: torch.empty(s, dtype=t, device=p.device)  # noqa: E731
        if codes is None:
            codes = new(p.out_elems, t=torch.int8)
        decode(p, compressed, codes, OUT_CODES, None, chunk_status)
        r = p.tensors[0]
        o, s = int(r["out_elem_offset"]), int(r["scale_row_offset"])
        w, ws = codes.view(-1)[o:o + v * d].view(v, d), scales.view(-1)[s:s + v]
        n = min(m, tokens)
        q, sx, logits = new(n, d, t=torch.int8), new(n), new(n, v)
        if dx is not None or dscales is not None:
            dlogits = new(n, v, t=x.dtype)
        if dscales is not None:
            sums, part = dscales.view(-1)[s:s + v].zero_(), new(v)
        for i in range(0, m, tokens):
            k = min(m - i, tokens)
            cut = lambda t: None if t is None else t[i:i + k]  # noqa: B023, E731
            entries = dict(teacher_lse=cut(teacher_lse), weight=cut(weight),
                           temperature=temperature)
            int8.quantize_rows(cut(x), q[:k], sx[:k])
            int8.gemm(q[:k], sx[:k], w, ws, logits[:k])
            if dx is None and dscales is None:
                distill.loss(logits[:k], cut(index), cut(teacher), cut(loss), **entries)
                continue
            distill.loss_backward(logits[:k], cut(index), cut(teacher), dlogits[:k], cut(dloss),
                                  cut(loss), **entries)
            # (a token that is not finite but has no weight takes no part in dscales)
            sx[:k].nan_to_num_()
            int8.gemm_backward(dlogits[:k], q[:k], sx[:k], w, ws, cut(dx),
                               part if dscales is not None else None)
            if dscales is not None:
                sums.add_(part)
