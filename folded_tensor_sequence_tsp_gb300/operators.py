"""Owners of the operators around a TSP layer, beside TSPLayer: each keeps the workspace
of its calls, sized once for the largest call, and allocates the outputs that the caller
does not bring.

One object serves one stream at a time: its calls share its workspace, so calls that may
overlap (two streams, two captured graphs that replay at the same time) need an object
each. A workspace that a captured graph may use is kept as long as its object lives, also where
TSPLinearE4M3.enable_backward() puts a larger one in its place. An object may serve another
stream than the one it was made on: its workspace is ready when the constructor returns. Like
any tensor, it is deleted once the streams it served are done with it.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple

import torch

from ._binding import (AdamW, TSP_OK, TSPError, _adamw_call, _adamw_check, _adamw_launch, _adamw_lists, _launch, _matrix, _rows, _same_device,
                       _scalar, tsp_device_status, tsp_grad_clip, tsp_grad_norm,
                       tsp_grad_workspace_bytes, tsp_last_error, tsp_matmul_e4m3_workspace_bytes, tsp_packed_attention_bwd,
                       tsp_packed_attention_fwd,
                       tsp_packed_attention_workspace_bytes, tsp_quantize_e4m3, tsp_rmsnorm_bwd, tsp_rmsnorm_fwd,
                       tsp_rmsnorm_fwd_e4m3, tsp_rmsnorm_workspace_bytes, tsp_status_init)

__all__ = ["TSPPackedAttention", "TSPRMSNorm", "TSPGradClip", "TSPWeightE4M3", "TSPLinearE4M3",
           "TSPAdamW"]


def _device(device):
    """The CUDA device of an object: the given one, by default the current one."""
    if isinstance(device, int):
        return torch.device("cuda", device)
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError(f"expected a CUDA device, got {device}")
    return device if device.index is not None else torch.device("cuda", torch.cuda.current_device())


def _on(stream, device):
    """Outputs made in here belong to the stream that the call runs on."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


def _not_in_a_capture(device, what):
    """What a constructor launches would become part of the graph instead of running now: an object
    with a status word and counters to zero is made before the capture."""
    with torch.cuda.device(device):
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError(f"{what} cannot be captured: call it before the capture begins")


def _ready(device):
    """Wait for what a constructor has queued, and for what its stream still has to do on memory
    that the constructor took over: the first call may come on another stream."""
    with torch.cuda.device(device):
        if not torch.cuda.is_current_stream_capturing():
            torch.cuda.current_stream(device).synchronize()


class TSPPackedAttention:
    """Causal attention over packed sequences with grouped heads: up to `tokens` rows in up to
    `n_seqs` sequences.

    q [T, heads, d], k and v [T, kv_heads, d] (bfloat16; rows may be strided, as column ranges
    of one projection are), starts int32 [n + 1] on the device: sequence s owns the rows
    starts[s] to starts[s + 1]. Rows outside every sequence are left as they were, in every
    output; outputs made here start as zeros."""

    def __init__(self, tokens, n_seqs, heads, kv_heads, head_dim, scale=None, device=None):
        self.tokens, self.n_seqs = tokens, n_seqs
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.scale = head_dim ** -0.5 if scale is None else float(scale)
        self.device = _device(device)
        _not_in_a_capture(self.device, "TSPPackedAttention()")
        nbytes = tsp_packed_attention_workspace_bytes(tokens, n_seqs, heads, kv_heads, head_dim)
        if nbytes == 0:
            raise TSPError(2, tsp_last_error())
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        tsp_status_init(self.ws)
        _ready(self.device)

    def _check(self, q, k, starts):
        if q.shape[1:] != (self.heads, self.head_dim) or k.shape[1:] != (self.kv_heads, self.head_dim):
            raise ValueError(f"made for {self.heads}/{self.kv_heads} heads of {self.head_dim}, got q "
                             f"{tuple(q.shape)} and k {tuple(k.shape)}")
        if q.shape[0] > self.tokens or starts.numel() - 1 > self.n_seqs:
            raise ValueError(f"made for {self.tokens} tokens in {self.n_seqs} sequences, got "
                             f"{q.shape[0]} in {starts.numel() - 1}")

    def _zeros(self, stream, *shape, dtype=torch.bfloat16):
        with _on(stream, self.device):
            return torch.zeros(shape, dtype=dtype, device=self.device)

    def forward(self, q, k, v, starts, out=None, stream=None):
        """o [T, heads, d]."""
        self._check(q, k, starts)
        if out is None:
            out = self._zeros(stream, *q.shape)
        tsp_packed_attention_fwd(q, k, v, starts, out, self.ws, None, self.scale, stream)
        return out

    def forward_train(self, q, k, v, starts, out=None, lse=None, stream=None):
        """(o, lse): forward() that also keeps the row statistics [heads, T] for backward()."""
        self._check(q, k, starts)
        if out is None:
            out = self._zeros(stream, *q.shape)
        if lse is None:
            lse = self._zeros(stream, self.heads, q.shape[0], dtype=torch.float32)
        tsp_packed_attention_fwd(q, k, v, starts, out, self.ws, lse, self.scale, stream)
        return out, lse

    def backward(self, q, k, v, starts, o, lse, dout, dq=None, dk=None, dv=None, stream=None):
        """(dq, dk, dv) from forward_train's o and lse and the gradient dout of o."""
        self._check(q, k, starts)
        dq = self._zeros(stream, *q.shape) if dq is None else dq
        dk = self._zeros(stream, *k.shape) if dk is None else dk
        dv = self._zeros(stream, *v.shape) if dv is None else dv
        tsp_packed_attention_bwd(q, k, v, starts, o, lse, dout, dq, dk, dv, self.ws, self.scale, stream)
        return dq, dk, dv

    def check(self, stream=None):
        """Synchronise and raise TSPError if the starts were out of order or a device wait gave up."""
        with torch.cuda.device(self.device):
            st = tsp_device_status(self.ws, stream)
        if st != TSP_OK:
            raise TSPError(st, tsp_last_error())


class TSPRMSNorm:
    """Residual addition and root-mean-square norm of up to `rows` rows of `width`.

    The weight is an argument of each call, so one object serves every norm of a stack
    with that width."""

    def __init__(self, rows, width, eps=1e-5, device=None):
        self.rows, self.width, self.eps = rows, width, eps
        self.device = _device(device)
        nbytes = tsp_rmsnorm_workspace_bytes(rows, width)
        if nbytes == 0:
            raise ValueError(f"TSPRMSNorm: unsupported size {rows} x {width}")
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        _ready(self.device)

    def _rows(self, t):
        """t as a [rows, width] matrix (None stays None)."""
        if t is None or (t.dim() == 2 and t.shape[1] == self.width):
            return t
        if t.dim() < 1 or t.shape[-1] != self.width:
            raise ValueError(f"expected rows of {self.width}, got shape {tuple(t.shape)}")
        return t.view(-1, self.width)

    def forward(self, x, weight, residual=None, y=None, h=None, stream=None):
        """(y, h): h = x + residual (None without a residual), y = norm(h) * weight in bf16."""
        with _on(stream, self.device):
            if y is None:
                y = torch.empty_like(x)
            if residual is not None and h is None:
                h = torch.empty_like(residual)
        v = self._rows
        tsp_rmsnorm_fwd(v(x), weight, v(y), v(residual), v(h), self.eps, stream)
        return y, h

    def forward_e4m3(self, x, weight, residual=None, group=128, y=None, scales=None, h=None,
                     stream=None):
        """(y, scales, h) with y in float8_e4m3fn; scales [rows, 1] for group 0, one per 128
        columns for group 128."""
        rows = x.numel() // self.width
        with _on(stream, self.device):
            if y is None:
                y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=x.device)
            if scales is None:
                scales = torch.empty((rows, -(-self.width // group) if group else 1),
                                     dtype=torch.float32, device=x.device)
            if residual is not None and h is None:
                h = torch.empty_like(residual)
        v = self._rows
        tsp_rmsnorm_fwd_e4m3(v(x), weight, v(y), scales, v(residual), v(h), self.eps, group,
                             stream)
        return y, scales, h

    def backward(self, h, weight, dy, dh=None, dx=None, dx16=None, dw=None, stream=None):
        """(dx, dw): the gradient of h (dh added when given) in h's type, and the weight's in
        fp32. h is forward's h, or its x when there was no residual."""
        if h.numel() > self.rows * self.width:
            raise ValueError(f"{h.numel() // self.width} rows; the workspace was made for {self.rows}")
        with _on(stream, self.device):
            if dx is None:
                dx = torch.empty_like(h)
            if dw is None:
                dw = torch.empty(self.width, dtype=torch.float32, device=h.device)
        v = self._rows
        tsp_rmsnorm_bwd(v(h), weight, v(dy), v(dx), dw, self.ws, v(dh), v(dx16), self.eps,
                        stream)
        return dx, dw


class TSPGradClip:
    """Global norm of up to `tensors` gradient tensors (fp32 and bf16 mixed), and clipping."""

    def __init__(self, tensors, device=None):
        nbytes = tsp_grad_workspace_bytes(tensors)
        if nbytes == 0:
            raise ValueError(f"TSPGradClip: unsupported number of tensors {tensors}")
        self.tensors = tensors
        self.device = _device(device)
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        _ready(self.device)

    def _norm(self, norm, stream):
        if norm is None:
            with _on(stream, self.device):
                norm = torch.empty((), dtype=torch.float32, device=self.device)
        return norm

    def norm(self, grads, norm=None, stream=None):
        """The 2-norm over all elements, as one float32 on the device."""
        norm = self._norm(norm, stream)
        tsp_grad_norm(grads, norm, self.ws, stream)
        return norm

    def clip(self, grads, max_norm, outs=None, norm=None, stream=None):
        """Scale the gradients to a global norm of at most max_norm, in place or into `outs`;
        returns the norm before scaling, as one float32 on the device."""
        norm = self._norm(norm, stream)
        tsp_grad_clip(grads, grads if outs is None else outs, float(max_norm), norm, self.ws, stream)
        return norm


class TSPWeightE4M3(NamedTuple):
    """A linear layer's weight [out, in] in 8 bits: values with a scale for 128 x 128 of them, and
    for the backward their transposes."""

    values: torch.Tensor
    scales: torch.Tensor
    values_t: torch.Tensor | None = None
    scales_t: torch.Tensor | None = None


def _blocks(n):
    return -(-n // 128)


def _up16(n):
    return -(-n // 16) * 16


class TSPLinearE4M3:
    """y = x w^T with products in e4m3: x and the gradients quantised per row and 128 columns (for dw
    along the tokens, per column and 128 tokens), w per 128 x 128 tile, sums in fp32. Up to `tokens`
    rows; the weight is an argument of each call."""

    def __init__(self, tokens, out_features, in_features, device=None):
        if tokens < 0 or out_features < 1 or in_features < 1:
            raise ValueError(f"TSPLinearE4M3: unsupported size {tokens} x {out_features} x {in_features}")
        self.tokens, self.out_features, self.in_features = tokens, out_features, in_features
        self.device = _device(device)
        _not_in_a_capture(self.device, "TSPLinearE4M3()")
        self._kept = []  # a workspace that growing replaced
        # byte offsets: status, then values and scales of x; of dy; of the transpose of dy
        self._at, at = [], tsp_matmul_e4m3_workspace_bytes()
        for rows, width in ((tokens, in_features), (tokens, out_features), (out_features, tokens)):
            self._at.append((at, at + _up16(width) * rows))
            at += _up16(width) * rows + -(-4 * rows * _blocks(width) // 256) * 256
            at = -(-at // 256) * 256
        self._sizes = (self._at[1][0], at)
        self._workspace(self._sizes[0])

    def _workspace(self, nbytes):
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        tsp_status_init(self.ws)
        _ready(self.device)

    def enable_backward(self):
        """Grow the workspace to the backward's size. Call it before capturing a training step; graphs
        captured before go on in the workspace that they were captured with, which is kept for them."""
        if self.ws.numel() < self._sizes[1]:
            _not_in_a_capture(self.device, "TSPLinearE4M3.enable_backward()")
            self._kept.append(self.ws)
            self._workspace(self._sizes[1])

    def quantize_weight(self, w, training=True, stream=None):
        """The TSPWeightE4M3 of w [out, in] (bfloat16 or float32), with its transpose for training."""
        n, k = self.out_features, self.in_features
        if w.shape != (n, k):
            raise ValueError(f"expected a weight [{n}, {k}], got {tuple(w.shape)}")
        with _on(stream, self.device):
            new = lambda r, c: torch.empty(r, _up16(c), dtype=torch.float8_e4m3fn, device=self.device)[:, :c]  # noqa: E731
            scale = lambda r, c: torch.empty(_blocks(r), _blocks(c), device=self.device)  # noqa: E731
            out = TSPWeightE4M3(new(n, k), scale(n, k), *((new(k, n), scale(k, n)) if training else ()))
        tsp_quantize_e4m3(w, *out, block=128, stream=stream)
        return out

    @staticmethod
    def _as_rows(x, width, name):
        """A [..., width] tensor as a matrix."""
        if x.dim() == 2:
            return x
        if x.dim() < 1 or x.shape[-1] != width:
            raise ValueError(f"{name}: expected rows of {width}, got shape {tuple(x.shape)}")
        return x.view(-1, width)

    def _input(self, x, width, name):
        """(rows, address, row stride) of a bfloat16 [..., width] tensor."""
        x = self._as_rows(x, width, name)
        if x.shape[0] > self.tokens:
            raise ValueError(f"{x.shape[0]} rows; the object was made for {self.tokens}")
        return x.shape[0], *_rows(x, name, (x.shape[0], width), (torch.bfloat16,))

    def _weight(self, values, scales, rows, width):
        if values is None:
            raise ValueError("the backward needs the weight's transpose: quantize_weight(w, training=True)")
        p, ld = _rows(values, "weight", (rows, width))
        return p, ld if rows > 1 else _up16(width), _matrix(scales, "weight scales", (_blocks(rows), _blocks(width)),
                                                            (torch.float32,))

    def _new(self, shape, dtype, stream):
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with _on(stream, self.device):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _out(self, out, shape, dtype, stream, name):
        if out is None:
            out = self._new(shape, dtype, stream)
        elif out.dtype != dtype or out.shape != shape or not out.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")
        return out

    def forward(self, x, weight, scales=None, out=None, stream=None):
        """y [..., out] in bfloat16. x [..., in]: bfloat16, or e4m3 [rows, in] with scales [rows, ceil(in / 128)]
        as TSPRMSNorm.forward_e4m3 (group 128) and tsp_quantize_e4m3 leave them, in rows that start on 16 bytes."""
        n, k = self.out_features, self.in_features
        device = _same_device((x, scales, *weight[:2], out, self.ws))
        out = self._out(out, (*x.shape[:-1], n), torch.bfloat16, stream, "out")
        w = self._weight(*weight[:2], n, k)
        ws = self.ws.data_ptr()
        if scales is None:
            m, xp, ldx = self._input(x, k, "x")
            if m:
                a, ld_a, sa = ws + self._at[0][0], _up16(k), ws + self._at[0][1]
                _launch("tsp_quantize_e4m3", device, stream, m, k, xp, 0, ldx, 1, a, ld_a, sa, None, 0, None)
        else:
            x = self._as_rows(x, k, "x")
            m = x.shape[0]
            a, ld_a = _rows(x, "x", (m, k))
            ld_a = ld_a if m > 1 else _up16(k)
            sa = _matrix(scales, "scales", (m, _blocks(k)), (torch.float32,))
        if m:
            _launch("tsp_matmul_e4m3", device, stream, m, n, k, a, ld_a, sa, *w, 128, out.data_ptr(), n, 0, 0, ws)
        return out

    def forward_train(self, x, weight, out=None, stream=None):
        """(y, saved): forward() of a bfloat16 x that also keeps what backward() needs of it, the transpose of
        x in 8 bits."""
        self.enable_backward()
        n, k = self.out_features, self.in_features
        device = _same_device((x, *weight[:2], out, self.ws))
        out = self._out(out, (*x.shape[:-1], n), torch.bfloat16, stream, "out")
        w = self._weight(*weight[:2], n, k)
        m, xp, ldx = self._input(x, k, "x")
        # the values [in, rows in a multiple of 16], then their scales [in, ceil(rows / 128)]
        kept = self._new((k * (_up16(m) + 4 * _blocks(m)),), torch.uint8, stream)
        if m:
            ws, xt = self.ws.data_ptr(), kept.data_ptr()
            a, ld_a, sa = ws + self._at[0][0], _up16(k), ws + self._at[0][1]
            _launch("tsp_quantize_e4m3", device, stream, m, k, xp, 0, ldx, 1, a, ld_a, sa, xt, _up16(m), xt + k * _up16(m))
            _launch("tsp_matmul_e4m3", device, stream, m, n, k, a, ld_a, sa, *w, 128, out.data_ptr(), n, 0, 0, ws)
        return out, (kept, m)

    def backward(self, saved, dy, weight, dx=None, dw=None, accumulate=False, stream=None):
        """(dx, dw) of forward_train's saved and the gradient dy [..., out] of y (bfloat16): dx in bfloat16, dw
        in float32, added to the given dw with accumulate."""
        self.enable_backward()
        n, k = self.out_features, self.in_features
        kept, rows = saved
        device = _same_device((dy, kept, *weight[2:], dx, dw, self.ws))
        m, gp, ldg = self._input(dy, n, "dy")
        if rows != m or kept.numel() != k * (_up16(m) + 4 * _blocks(m)):
            raise ValueError(f"saved belongs to {rows} rows of another layer or call, dy has {m}")
        wt = self._weight(*(weight[2:] or (None, None)), k, n)
        if accumulate and dw is None:
            raise ValueError("accumulate needs a dw to add to")
        dx = self._out(dx, (*dy.shape[:-1], k), torch.bfloat16, stream, "dx")
        dw = self._out(dw, (n, k), torch.float32, stream, "dw")
        ws = self.ws.data_ptr()
        g, sg, gt, sgt = (ws + at for pair in self._at[1:] for at in pair)
        if m:
            _launch("tsp_quantize_e4m3", device, stream, m, n, gp, 0, ldg, 1, g, _up16(n), sg, gt, _up16(m), sgt)
            _launch("tsp_matmul_e4m3", device, stream, m, k, n, g, _up16(n), sg, *wt, 128, dx.data_ptr(), k, 0, 0, ws)
        xt = kept.data_ptr()
        _launch("tsp_matmul_e4m3", device, stream, n, k, m, gt, _up16(m), sgt, xt, _up16(m), xt + k * _up16(m), 1,
                dw.data_ptr(), k, 1, int(accumulate), ws)
        return dx, dw

    def check(self, stream=None):
        """Synchronise and raise TSPError if a bounded device wait gave up."""
        with torch.cuda.device(self.device):
            for ws in (self.ws, *self._kept):
                st = tsp_device_status(ws, stream)
                if st != TSP_OK:
                    raise TSPError(st, tsp_last_error())


class TSPAdamW:
    """AdamW over a list of float32 and bfloat16 weights, updated in place.

    masters: for each bfloat16 weight a float32 tensor that holds it exactly, or None (the weight is
    then rounded stochastically). The states are made here, as zeros: float32, or with state_bits 8
    float8_e4m3fn with a float32 scale for each 128 elements. The object keeps the addresses of weights,
    masters and states: they are updated where they are, and may not be replaced."""

    def __init__(self, params, masters=None, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.0, state_bits=32, seed=0,
                 device=None):
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        self.params, self.masters = list(params), None if masters is None else list(masters)
        self.betas, self.eps, self.weight_decay, self.seed = betas, eps, weight_decay, seed
        self.state_bits = state_bits
        self.device = _device(self.params[0].device if self.params and device is None else device)
        if any(p.device != self.device for p in self.params):
            raise ValueError(f"the weights must be on {self.device}")
        if self.masters is not None and any(m is not None and p.dtype != torch.bfloat16
                                            for m, p in zip(self.masters, self.params)):
            raise ValueError("a master belongs beside a bfloat16 weight")
        _not_in_a_capture(self.device, "TSPAdamW()")
        kind = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        new = lambda n, dtype: torch.zeros(n, dtype=dtype, device=self.device)  # noqa: E731
        sizes = [p.numel() for p in self.params]
        scales = [[new(-(-n // 128), torch.float32) for n in sizes] if state_bits == 8 else None for _ in range(2)]
        self.resume(0, [new(n, kind) for n in sizes], [new(n, kind) for n in sizes], *scales)
        _ready(self.device)

    def resume(self, t, m, v, m_scales=None, v_scales=None):
        """Go on after t steps with these states (of the types and sizes that the constructor makes),
        which are taken over, not copied."""
        if (m_scales is not None) != (self.state_bits == 8):
            raise ValueError("scales belong to states of 8 bits")
        lists = _adamw_lists(self.params, self.masters, m, v, m_scales, v_scales)
        self.t, self.m, self.v, self.m_scales, self.v_scales = t, m, v, m_scales, v_scales
        self._lists = lists

    def _call(self, grads, lr, norm, max_norm, t):
        device = self.device.index
        step = AdamW(0.0, *self.betas, self.eps, self.weight_decay, max_norm, self.t + 1, self.seed & 0xFFFFFFFF,
                     _scalar(norm, "norm", torch.float32, device), None, None)
        if isinstance(lr, torch.Tensor):
            step.device_lr = _scalar(lr, "lr", torch.float32, device)
        else:
            step.lr = lr
        if t is not None:
            step.device_t = _scalar(t, "t", torch.int64, device)
        return _adamw_call(self._lists, grads, step)

    def _run(self, call, t, stream):
        _adamw_launch(call, stream)
        if t is None:
            self.t += 1

    def step(self, grads, lr, norm=None, max_norm=float("inf"), t=None, stream=None):
        """One step with the gradients of all weights (None: that weight is left as it is).

        norm: the gradients' global norm, one float32 on the device (TSPGradClip.norm); they are
        then scaled to a norm of at most max_norm on the way. lr may be one float32 on the device,
        and t one int64, this step's number from 1, in place of the object's own count: a captured
        step is then replayed with their values of that moment."""
        self._run(self._call(grads, lr, norm, max_norm, t), t, stream)


def _step_together(optimizers, parts, lr, norm, max_norm, t, stream=None):
    """A step of each optimizer with its part of the gradients, or, where one refuses, of none."""
    calls = [o._call(part, lr, norm, max_norm, t) for o, part in zip(optimizers, parts)]
    for call in calls[1:]:  # the first step refuses before anything runs
        _adamw_check(call)
    for optimizer, call in zip(optimizers, calls):
        optimizer._run(call, t, stream)
