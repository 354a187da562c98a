"""A transformer's feed-forward block on compressed Int8 weights:

    y = (act(x . gate^T) * (x . up^T)) . down^T

The three matrices are one plan (Int8 tensors in the order gate, up, down).
They are decoded to codes right before the block uses them [EntQuant,
"Float8@2bits ...", technical summary §2 "Decodificación en Tiempo de
Inferencia"] and multiplied as codes: activations are quantised to int8 per
row, both first products and the activation are one kernel, and its result is
quantised again for the last product. The backward pass gives the gradients
of x and of every row scale; the codes are constants. Neither records an
autograd graph, and an x or dy that would need one is refused: a
torch.autograd.Function calls ``forward`` and ``backward`` for it.

``residual`` is the block between its norms, as it stands in a transformer,

    out = alpha x + beta gate norm(block(norm(x) pre)) post

with the first norm written as the codes that the products take and the rest in
one kernel; ``residual_backward`` gives its gradients.
"""
from __future__ import annotations

import contextlib
import weakref

import torch

from . import EINVAL, KIND_INT8, OUT_CODES, EntqError, Plan, _device_buffer, decode, int8, norm


def _on(stream, device):
    """Makes ``stream`` (torch stream, raw handle or None) the current one."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=device) if stream
                  else torch.cuda.default_stream(device))
    return torch.cuda.stream(stream)


class _Memory:
    """Orders the use of memory that was allocated on the stream ``home`` with
    what home's allocator does with it before and after: work on another
    stream starts after what home had queued when it was allocated, and home
    waits for the last such work when the memory goes back to it. (Events, not
    record_stream: a caller's raw stream may be gone by then.)"""

    def __init__(self, owner, home):
        self.home, self.ends = home, {}
        self.begin = home.record_event()
        weakref.finalize(owner, self.give_back, home, self.ends).atexit = False

    @staticmethod
    def give_back(home, ends):
        for end in ends.values():
            home.wait_event(end)

    @contextlib.contextmanager
    def on(self, stream):
        if stream == self.home or torch.cuda.is_current_stream_capturing():
            # (a capture cannot wait for events from outside it; torch.cuda.graph
            # starts one after all work queued before has ended)
            yield
            return
        stream.wait_event(self.begin)
        try:
            yield
        finally:
            self.ends.setdefault(stream.cuda_stream, torch.cuda.Event()).record(stream)


class DecodedCodes:
    """The code buffer of a block of Int8 tensors: its checks, its decode, and
    the order of its use on several streams."""

    def __init__(self, p: Plan, scales, codes):
        _device_buffer(p, "scales", scales, p.scale_rows, dtypes=(torch.float32,))
        self._memory = None
        if codes is None:
            codes = torch.empty(p.out_elems, dtype=torch.int8, device=p.device)
            if not torch.cuda.is_current_stream_capturing():
                self._memory = _Memory(self, torch.cuda.current_stream(p.device))
        _device_buffer(p, "codes", codes, p.out_elems, dtypes=(torch.int8,))
        self.plan, self.scales, self.codes = p, scales, codes

    @contextlib.contextmanager
    def _using_codes(self, stream):
        """Makes ``stream`` the current one for work on the code buffer."""
        with _on(stream, self.plan.device):
            if self._memory is None:
                yield
            else:
                with self._memory.on(torch.cuda.current_stream(self.plan.device)):
                    yield

    def decode(self, compressed, chunk_status=None, stream=None):
        """Enqueue the decode of the block's codes."""
        with self._using_codes(stream):
            decode(self.plan, compressed, self.codes, OUT_CODES, None, chunk_status)


class FeedForward(DecodedCodes):
    """p: the plan of gate [F, D], up [F, D] and down [E, F]; scales: device
    float32 with the plan's row scales. ``decode`` fills the code buffer, which
    ``forward`` and ``backward`` then use; a caller that walks over layers gives
    several blocks one buffer (``codes``: device int8, at least out_elems).
    hidden_type: the type of the hidden values between the products, which are
    quantised again at once; None: x's type. In float16 a hidden value beyond
    65,504 is an infinity, which makes its token NaN; torch.float32 has
    neither that limit nor a rounding before the quantiser's.
    Every call may run on a stream of its own. The caller orders them (a decode
    before the products that use it); a buffer that the block allocated itself
    needs no further care, but a block that a graph captured has to outlive
    the graph."""

    def __init__(self, p: Plan, scales, activation="silu", codes=None, hidden_type=None):
        t = p.tensors
        if p.n_tensors != 3 or any(int(k) & 0xFF != KIND_INT8 for k in t["kind"]):
            raise EntqError(EINVAL, "a feed-forward block is three Int8 tensors: gate, up, down")
        (f, d), (f2, d2), (e, f3) = ((int(r["rows"]), int(r["cols"])) for r in t)
        if (f, d) != (f2, d2) or f3 != f:
            raise EntqError(EINVAL, f"gate {f} x {d}, up {f2} x {d2}, down {e} x {f3}: gate and "
                                    "up have one shape, down a column for each of their rows")
        if max(d, f) > int8.MAX_COLS:
            raise EntqError(EINVAL, f"{max(d, f)} columns, at most {int8.MAX_COLS} are taken")
        if activation not in int8.ACTIVATIONS:
            raise EntqError(EINVAL, f"activation {activation!r}: one of "
                                    f"{', '.join(int8.ACTIVATIONS)}")
        if hidden_type not in (None, torch.bfloat16, torch.float16, torch.float32):
            raise EntqError(EINVAL, f"hidden values of type {hidden_type}")
        super().__init__(p, scales, codes)
        self.activation = activation
        self.width, self.hidden, self.out = d, f, e
        self.hidden_type = hidden_type
        self._w = []  # code matrix and its scales
        self._at = []  # where a tensor's scales are
        codes, scales = self.codes.view(-1), scales.view(-1)
        for r in t:
            rows, cols = int(r["rows"]), int(r["cols"])
            o, s = int(r["out_elem_offset"]), int(r["scale_row_offset"])
            self._at.append(slice(s, s + rows))
            self._w += [codes[o:o + rows * cols].view(rows, cols), scales[s:s + rows]]

    def forward(self, x, y, stream=None):
        """y = block(x): x bfloat16, float16 or float32 [m, D], y of any of
        these types [m, E]."""
        index = self.plan.device.index
        m = int8._check_activations("x", x, index, self.width)
        int8._check_result("y", y, index, m, self.out)
        with self._using_codes(stream):
            h = torch.empty(m, self.hidden, dtype=self.hidden_type or x.dtype, device=x.device)
            int8.gated(x, None, *self._w[:4], h, self.activation)
            int8.gemm(h, None, *self._w[4:], y)

    def backward(self, dy, x, dx=None, dscales=None, stream=None):
        """Gradients for dy = dL/dy (bfloat16 or float16 [m, E], x's type):
        dx (that type, [m, D]) and dscales (float32 [scale_rows], the plan's
        order); None: not computed. The forward pass is done again from x."""
        index = self.plan.device.index
        m = int8._check_activations("x", x, index, self.width, (int8._BF16, int8._F16))
        int8._grad_rows("dy", dy, index, m, self.out)
        if x.dtype != dy.dtype:
            raise EntqError(EINVAL, f"dy has dtype {dy.dtype}, x {x.dtype}")
        if dx is not None:
            int8._matrix("dx", dx, index, (int8._TYPES[x.dtype],), (m, self.width))
        if dscales is not None:
            _device_buffer(self.plan, "dscales", dscales, self.plan.scale_rows,
                           dtypes=(torch.float32,))
        with self._using_codes(stream):
            q = torch.empty(m, self.width, dtype=torch.int8, device=x.device)
            sx = torch.empty(m, dtype=torch.float32, device=x.device)
            int8.quantize_rows(x, q, sx)
            h = self._hidden(q, sx, x.dtype)
            self._backward(dy, q, sx, *h, dx, dscales)

    def _hidden(self, q, sx, dtype):
        """The hidden values' codes and scales."""
        m = q.shape[0]
        h = torch.empty(m, self.hidden, dtype=self.hidden_type or dtype, device=q.device)
        qh = torch.empty(m, self.hidden, dtype=torch.int8, device=q.device)
        sh = torch.empty(m, dtype=torch.float32, device=q.device)
        int8.gated(q, sx, *self._w[:4], h, self.activation)
        int8.quantize_rows(h, qh, sh)
        return qh, sh

    def _backward(self, dy, q, sx, qh, sh, dx, dscales):
        dh = torch.empty(q.shape[0], self.hidden, dtype=dy.dtype, device=dy.device)
        dg, du, dd = (dscales.view(-1)[s] if dscales is not None else None for s in self._at)
        int8.gemm_backward(dy, qh, sh, *self._w[4:], dh, dd)
        int8.gated_backward(dh, q, sx, *self._w[:4], dx, dg, du, self.activation)

    def _check_residual(self, x, pre, post, gate, alpha, beta, eps):
        if self.out != self.width:
            raise EntqError(EINVAL, f"a residual block has as many results as columns, this one "
                                    f"{self.out} and {self.width}")
        index = self.plan.device.index
        int8._check_activations("x", x, index, self.width)
        # (x in the place of the block's result, which has its shape and type)
        if pre is None:
            raise EntqError(EINVAL, "pre is required")
        return norm._describe(x, x, post, gate, pre, alpha, beta, eps)

    def residual(self, x, out, pre, post=None, gate=None, alpha=1.0, beta=1.0, eps=1e-6,
                 stream=None):
        """out = alpha x + beta gate norm(block(norm(x) pre)) post: x and out
        bfloat16, float16 or float32 [m, D] of one type (out may be x), the
        rest as in ``norm.block``; without post the block's result is not
        normalised."""
        index, a = self._check_residual(x, pre, post, gate, alpha, beta, eps)
        int8._matrix("out", out, index, (a.type,), x.shape)
        with self._using_codes(stream):
            q, sx = self._normed(x, pre, eps)
            y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
            h = torch.empty(x.shape[0], self.hidden, dtype=self.hidden_type or x.dtype,
                            device=x.device)
            int8.gated(q, sx, *self._w[:4], h, self.activation)
            int8.gemm(h, None, *self._w[4:], y)
            norm.block(x, y, out, post, gate, alpha=alpha, beta=beta, eps=eps)

    def _normed(self, x, pre, eps):
        q = torch.empty(x.shape, dtype=torch.int8, device=x.device)
        sx = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        norm.block(x, pre=pre, y=q, y_scales=sx, eps=eps)
        return q, sx

    def residual_backward(self, dout, x, pre, post=None, gate=None, dx=None, dscales=None,
                          dpre=None, dpost=None, dgate=None, alpha=1.0, beta=1.0, eps=1e-6,
                          stream=None):
        """Gradients of ``residual`` for dout = dL/dout (bfloat16 or float16
        [m, D], x's type): dx (that type), dscales (float32 [scale_rows]),
        dpre, dpost (float32 [D]) and dgate (as the gate); None: not computed.
        The forward pass is done again from x. Where alpha is not 1, alpha dout
        is rounded to dout's type before the rest of dx is added."""
        index, a = self._check_residual(x, pre, post, gate, alpha, beta, eps)
        int8._matrix("x", x, index, (int8._BF16, int8._F16))
        int8._grad_rows("dout", dout, index, *x.shape)
        if x.dtype != dout.dtype:
            raise EntqError(EINVAL, f"dout has dtype {dout.dtype}, x {x.dtype}")
        if dx is not None:
            int8._matrix("dx", dx, index, (a.type,), x.shape)
        if dscales is not None:
            _device_buffer(self.plan, "dscales", dscales, self.plan.scale_rows,
                           dtypes=(torch.float32,))
        for name, t, of in (("dpre", dpre, pre), ("dpost", dpost, post)):
            if t is not None:
                if of is None:
                    raise EntqError(EINVAL, f"{name} without {name[1:]}")
                int8._vector(name, t, index, self.width)
        if dgate is not None:
            if gate is None or norm._gate("dgate", dgate, a.type, index, *x.shape)[0] != a.gate_kind:
                raise EntqError(EINVAL, "dgate goes with a gate of its shape")
        with self._using_codes(stream):
            q, sx = self._normed(x, pre, eps)
            h = self._hidden(q, sx, x.dtype)
            new = lambda: torch.empty(x.shape, dtype=x.dtype, device=x.device)  # noqa: E731
            y, dy, dn = new(), new(), new()
            int8.gemm(*h, *self._w[4:], y)
            rest = dout if alpha == 1 else new()
            norm.block_backward(x, dout, None, y, post, gate, None, None if alpha == 1 else rest,
                                dy, dgate, None, dpost, alpha, beta, eps)
            if dx is None and dpre is None and dscales is None:
                return
            wanted = dx is not None or dpre is not None
            self._backward(dy, q, sx, *h, dn if wanted else None, dscales)
            if wanted:
                norm.block_backward(x, rest, dn, pre=pre, dx=dx, dpre=dpre, eps=eps)
