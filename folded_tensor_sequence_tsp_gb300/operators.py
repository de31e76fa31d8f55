"""Owners of the operators around a TSP layer, beside TSPLayer: each keeps the workspace
of its calls, sized once for the largest call, and allocates the outputs that the caller
does not bring.

One object serves one stream at a time: its calls share its workspace, so calls that may
overlap (two streams, two captured graphs that replay at the same time) need an object
each. The workspace is never replaced, so a captured graph stays valid as long as its
object lives. An object may serve another stream than the one it was made on: its workspace is
ready when the constructor returns. Like any tensor, it is deleted once the streams it served
are done with it.
"""
from __future__ import annotations

import contextlib

import torch

from ._binding import (TSP_OK, TSPError, tsp_device_status, tsp_grad_clip, tsp_grad_norm,
                       tsp_grad_workspace_bytes, tsp_last_error, tsp_packed_attention_bwd,
                       tsp_packed_attention_fwd,
                       tsp_packed_attention_workspace_bytes, tsp_rmsnorm_bwd, tsp_rmsnorm_fwd,
                       tsp_rmsnorm_fwd_e4m3, tsp_rmsnorm_workspace_bytes, tsp_status_init)

__all__ = ["TSPPackedAttention", "TSPRMSNorm", "TSPGradClip"]


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
