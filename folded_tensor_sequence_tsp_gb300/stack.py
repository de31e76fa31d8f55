"""A stack of pre-norm TSP layers: forward, training forward, backward and clipping.

Per layer, on the sharded activations ([D, S/D, H], or [D, batch, S/D, H]):
    a = Attn(norm(h) w_attn),  h += a
    m = MLP(norm(h) w_mlp),    h += m
and a last norm behind the last layer. The blocks are tsp_attention_fwd / tsp_mlp_fwd,
which return without a residual; the residual's addition, the rounding of the stream and
the next norm are one pass (tsp_rmsnorm_fwd). The stream h is kept in fp32 by default. All
layers share one plan and one workspace. Like the operators' objects, a stack serves one stream
at a time. Calls run on the stack's device, on the stream that is current there.
"""
from __future__ import annotations

import functools

import torch

from ._binding import (TSP_OK, TSPError, tsp_attention_bwd, tsp_attention_fwd, tsp_bwd_workspace_bytes,
                       tsp_device_status, tsp_last_error, tsp_mlp_bwd, tsp_mlp_fwd, tsp_pack_weights,
                       tsp_packed_weight_bytes, tsp_plan, tsp_plan_batched, tsp_workspace_bytes,
                       tsp_workspace_init)
from .operators import TSPGradClip, TSPRMSNorm, _device, _not_in_a_capture, _ready

__all__ = ["TSPStack"]

_MATRICES = ("Wq", "Wk", "Wv", "Wo", "W1", "W3", "W2")
_NORMS = ("attn_norm", "mlp_norm")


def _on_its_device(method):
    """The layer's calls launch on the current device, whatever device their tensors are on."""
    @functools.wraps(method)
    def call(self, *args, **kwargs):
        with torch.cuda.device(self.device):
            return method(self, *args, **kwargs)
    return call


class TSPStack:
    """weights: one dict per layer with Wq, Wk, Wv, Wo, W1, W3, W2 (bfloat16 CUDA tensors,
    nn.Linear layout) and the norm weights attn_norm and mlp_norm [hidden]; last_norm [hidden]; all
    on `device` (by default the current one)."""

    def __init__(self, D, S, hidden, heads, ffn, weights, last_norm, eps=1e-5, batch=1,
                 stream_dtype=torch.float32, device=None):
        if stream_dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("stream_dtype must be float32 or bfloat16")
        self.device = _device(device)
        _not_in_a_capture(self.device, "TSPStack()")
        if any(t.device != self.device for t in [last_norm, *(w[k] for w in weights for k in _MATRICES + _NORMS)]):
            raise ValueError(f"the weights must be on {self.device}")
        self.plan = (tsp_plan(D, S, hidden, heads, ffn) if batch == 1
                     else tsp_plan_batched(D, S, batch, hidden, heads, ffn))
        self.stream_dtype = stream_dtype
        self.wpack = []
        self._kept = []  # a workspace that growing replaced
        self._pack(weights)
        # the norm in front of each block, and the last one
        self.norms = [w[k] for w in weights for k in _NORMS] + [last_norm]
        self.norm = TSPRMSNorm(self.plan.info.tokens, hidden, eps, device=self.device)
        self.clipper = TSPGradClip(len(self.wpack) + len(self.norms), device=self.device)

    @_on_its_device
    def _pack(self, weights):
        for w in weights:
            packed = torch.empty(tsp_packed_weight_bytes(self.plan) // 2, dtype=torch.bfloat16,
                                 device=self.device)
            tsp_pack_weights(self.plan, *(w[k] for k in _MATRICES), packed)
            self.wpack.append(packed)
        self._workspace(tsp_workspace_bytes(self.plan))

    def _workspace(self, nbytes):
        self.ws = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
        tsp_workspace_init(self.plan, self.ws)
        _ready(self.device)

    @_on_its_device
    def enable_backward(self):
        """Grow the workspace to the backward's size (it serves the forward too). Call it before
        capturing a training step. Graphs of the forward captured before it go on in the workspace
        that they were captured with, which is kept for them."""
        need = tsp_bwd_workspace_bytes(self.plan)
        if self.ws.numel() < need:
            _not_in_a_capture(self.device, "TSPStack.enable_backward()")
            self._kept.append(self.ws)
            self._workspace(need)

    @property
    def shape(self):
        i = self.plan.info
        return (i.D, i.T, i.hidden) if i.batch == 1 else (i.D, i.batch, i.T, i.hidden)

    def _blocks(self):
        """(layer, forward, backward) of every block in order."""
        for layer in range(len(self.wpack)):
            yield layer, tsp_attention_fwd, tsp_attention_bwd
            yield layer, tsp_mlp_fwd, tsp_mlp_bwd

    def _run(self, xs, keep):
        h = xs if self.stream_dtype == xs.dtype else xs.to(self.stream_dtype)
        y, _ = self.norm.forward(xs, self.norms[0])
        for i, (layer, forward, _) in enumerate(self._blocks()):
            block = torch.empty(self.shape, dtype=torch.bfloat16, device=self.device)
            forward(self.plan, y, self.wpack[layer], block, self.ws)
            if keep is not None:
                keep.append((y, h))
                y, h = self.norm.forward(block, self.norms[i + 1], residual=h)
            else:
                # nothing of the last step is kept: the norm goes over the block's output, and
                # the stream over itself (but for the caller's xs)
                y, h = self.norm.forward(block, self.norms[i + 1], residual=h, y=block,
                                         h=None if h is xs else h)
        if keep is not None:
            keep.append((y, h))
        return y

    @_on_its_device
    def forward(self, xs):
        """The normed output of the stack for the sharded bfloat16 input xs."""
        return self._run(xs.view(self.shape), None)

    @_on_its_device
    def forward_train(self, xs):
        """(output, saved): forward() that keeps each block's input and the stream."""
        self.enable_backward()
        saved = []
        return self._run(xs.view(self.shape), saved), saved

    @_on_its_device
    def backward(self, saved, dout):
        """(dxs, grads) of the output gradient dout: dxs in the stream's type; grads is one
        packed fp32 weight gradient per layer (see tsp_unpack_weight_grads), then one fp32
        gradient per norm in the order attn_norm, mlp_norm of every layer, last_norm."""
        self.enable_backward()
        info = self.plan.info
        dpacked = [torch.empty(info.wpack_elems, dtype=torch.float32, device=self.device)
                   for _ in self.wpack]
        dnorms = [None] * len(self.norms)
        f32 = self.stream_dtype == torch.float32

        def through_norm(i, dy, dh):
            """Gradient of the stream in front of norm i, and its bfloat16 copy for the block."""
            h = saved[i][1]
            d16 = torch.empty(self.shape, dtype=torch.bfloat16, device=self.device) if f32 else None
            dx, dnorms[i] = self.norm.backward(h, self.norms[i], dy, dh=dh, dx=dh, dx16=d16)
            return dx, d16 if f32 else dx

        dh, dblock = through_norm(len(self.norms) - 1, dout.view(self.shape), None)
        for i, (layer, _, backward) in reversed(list(enumerate(self._blocks()))):
            dy = torch.empty(self.shape, dtype=torch.bfloat16, device=self.device)
            backward(self.plan, saved[i][0], self.wpack[layer], dblock, dy, dpacked[layer], self.ws)
            dh, dblock = through_norm(i, dy, dh)
        return dh, dpacked + dnorms

    @_on_its_device
    def clip(self, grads, max_norm):
        """Scale backward()'s grads in place to a global norm of at most max_norm; returns the
        norm as one float32 on the device. The packed layout's padding holds zeros."""
        return self.clipper.clip(grads, max_norm)

    @_on_its_device
    def check(self):
        """Synchronise and raise TSPError if a bounded device wait gave up."""
        for ws in (self.ws, *self._kept):
            st = tsp_device_status(ws)
            if st != TSP_OK:
                raise TSPError(st, tsp_last_error())
