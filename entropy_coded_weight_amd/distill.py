"""The distillation loss of a compressed model's logits against its teacher's
top logits, and the gradient that trains the row scales (the entq_distill_*
calls of include/entq.h): what goes before ``int8.gemm_backward`` of the output
projection. ``linear.distill_int8`` runs both over many tokens.

For token m with z = logits[m] / T, q = softmax(z) and the teacher's p over
the classes index[m]:

    loss[m] = weight[m] sum_j p_j (log p_j - log q_(index j))

p is the softmax of teacher[m] / T over the token's entries, or, with
``teacher_lse`` (the logsumexp of all the teacher's logits / T), exp(teacher /
T - lse), and the mass outside the entries is compared with the student's mass
there as one more class. An index below 0 is no entry; a row of weight 0 may
hold anything. Masks may be the type's lowest value or -infinity. A NaN in a
token's logits, entries or log-sum, or an index beyond the classes, makes all of
its loss and gradient NaN.

logits: bfloat16, float16 or float32 [M, V]; index: int32 or int64 [M, K], K
up to MAX_TOP; teacher: any of the logits' types [M, K] (unit stride along the
rows of each); teacher_lse and weight: float32 [M]. Streams, and what needs an
autograd graph, are as in ``int8``.
"""
from __future__ import annotations

import torch

from . import EINVAL, Distill, EntqError, lib
from .int8 import _BF16, _F16, _F32, _TYPES, _enqueue, _gpu, _matrix, _no_graph, _vector
from .norm import _number

MAX_TOP = 256
MAX_CLASSES = 262144

_FLOATS = (_BF16, _F16, _F32)


def _index(t, index, shape):
    """(bytes, row stride) of the indices."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index:
        raise EntqError(EINVAL, f"index: a torch tensor on cuda:{index} is required")
    if t.dtype not in (torch.int32, torch.int64) or t.shape != shape:
        raise EntqError(EINVAL, f"index: {t.dtype} {tuple(t.shape)}; int32 or int64 "
                                f"{tuple(shape)} is required")
    ld = t.stride(0) if shape[0] > 1 else max(t.stride(0), shape[1])
    if (t.stride(1) != 1 and shape[1] > 1) or ld < shape[1]:
        raise EntqError(EINVAL, f"index: strides {t.stride()}; rows of unit stride that do not "
                                "overlap are required")
    return t.element_size(), ld


def _describe(logits, index, teacher, teacher_lse, weight, temperature):
    dev = _gpu("logits", logits)
    kind, ld = _matrix("logits", logits, dev, _FLOATS)
    _no_graph("logits", logits)
    return dev, _entries(dev, *logits.shape, kind, logits.data_ptr(), ld, index, teacher,
                         teacher_lse, weight, temperature)


def _entries(dev, m, v, kind, z, ld, index, teacher, teacher_lse, weight, temperature):
    """The call for m x v logits of type ``kind`` at z."""
    if not 1 <= v <= MAX_CLASSES:
        raise EntqError(EINVAL, f"{v} classes, 1 to {MAX_CLASSES} are taken")
    if not isinstance(teacher, torch.Tensor) or teacher.dim() != 2 or teacher.shape[0] != m:
        raise EntqError(EINVAL, f"teacher: a matrix with a row for each of {m} tokens is required")
    k = teacher.shape[1]
    if not 1 <= k <= MAX_TOP:
        raise EntqError(EINVAL, f"{k} entries for each token, 1 to {MAX_TOP} are taken")
    tkind, ldt = _matrix("teacher", teacher, dev, _FLOATS)
    _no_graph("teacher", teacher)
    size, ldi = _index(index, dev, teacher.shape)
    lse = 0 if teacher_lse is None else _vector("teacher_lse", teacher_lse, dev, m)
    w = 0 if weight is None else _vector("weight", weight, dev, m)
    t = _number("temperature", temperature)
    if not 1e-4 <= t <= 1e4:
        raise EntqError(EINVAL, f"temperature {t}: 1e-4 to 1e4 is taken")
    return Distill(m, v, k, kind, tkind, size, t, 0, z, index.data_ptr(), teacher.data_ptr(), ld,
                   ldi, ldt, lse, w)


def loss(logits, index, teacher, loss, teacher_lse=None, weight=None, temperature=1.0,
         stream=None):
    """The tokens' losses into ``loss`` (float32 [M])."""
    dev, d = _describe(logits, index, teacher, teacher_lse, weight, temperature)
    p = _vector("loss", loss, dev, d.rows)
    _enqueue("entq_distill_loss", lambda w, n, s: lib().entq_distill_loss(d, p, s), 0, dev, stream,
             None)


def loss_backward(logits, index, teacher, dlogits, dloss=None, loss=None, teacher_lse=None,
                  weight=None, temperature=1.0, stream=None):
    """The gradient of sum(dloss * loss) (dloss float32 [M]; None: all 1) into
    ``dlogits`` (the logits' type [M, V], or of float32 logits any of the
    types, as ``int8.gemm_backward`` takes 16 bits; it overlaps nothing), and,
    unless None, the losses into ``loss``: a training step needs no call of
    ``loss`` before, and the logits are read once for both (rows of more than
    130,560 classes of 16 bits or 65,280 of float32 three times, and two times
    by ``loss``)."""
    dev, d = _describe(logits, index, teacher, teacher_lse, weight, temperature)
    kind, ld = _matrix("dlogits", dlogits, dev, _FLOATS if d.type == _F32 else (d.type,),
                       logits.shape)
    g = 0 if dloss is None else _vector("dloss", dloss, dev, d.rows)
    p = 0 if loss is None else _vector("loss", loss, dev, d.rows)
    _enqueue("entq_distill_backward",
             lambda w, n, s: lib().entq_distill_backward(d, g, dlogits.data_ptr(), kind, ld, p,
                                                          s), 0, dev, stream, None)
