"""Thin ctypes binding of libtsp.so (declared in include/tsp.h).

Argument marshalling only: each function checks the tensors it is given (device,
dtype, contiguity, size - the C ABI takes raw pointers and cannot check sizes),
passes their pointers and the current CUDA stream, and raises TSPError on a
non-OK status. Every step of the computation runs in the library's kernels; if
the library is not built, loading fails loudly.
"""
from __future__ import annotations

import array
import ctypes
import os
import re

import torch

from . import build as _build

__all__ = [
    "TSPError", "PlanInfo", "Plan", "load_library", "library_path", "declared_functions",
    "TSP_OK", "TSP_ERR_INVALID_ARG", "TSP_ERR_UNSUPPORTED", "TSP_ERR_CUDA", "TSP_ERR_TIMEOUT",
    "tsp_plan", "tsp_plan_batched", "tsp_get_plan_info", "tsp_workspace_bytes", "tsp_packed_weight_bytes",
    "tsp_workspace_init", "tsp_pack_weights", "tsp_shard_index", "tsp_shard", "tsp_unshard",
    "tsp_attention_fwd", "tsp_mlp_fwd", "tsp_mlp_fwd_noalloc", "tsp_layer_fwd", "tsp_layer_fwd_host",
    "tsp_qkv_projection", "tsp_qkv_projection_gathered", "tsp_kv_allgather",
    "tsp_causal_attention", "tsp_causal_attention_q", "tsp_o_projection",
    "tsp_swiglu_gate_up", "tsp_swiglu_down", "tsp_device_status", "tsp_wait_selftest",
    "tsp_last_error", "tsp_bwd_workspace_bytes", "tsp_mlp_bwd", "tsp_unpack_weight_grads",
    "tsp_attention_bwd", "tsp_layer_bwd", "tsp_causal_attention_lse", "tsp_causal_attention_bwd",
    "SCHEMES", "tsp_cost_model", "tsp_cost_model_batched", "tsp_cost_max_batch", "tsp_saved_bytes", "tsp_layer_fwd_train", "tsp_layer_bwd_saved",
    "tsp_rank_shard_bytes", "tsp_pack_rank_shard", "tsp_rank_qkv", "tsp_rank_kv_gather",
    "tsp_rank_attention", "tsp_rank_o_accumulate", "tsp_rank_mlp_step",
    "tsp_packed_attention_workspace_bytes", "tsp_status_init", "tsp_packed_attention_fwd",
    "tsp_packed_attention_bwd", "tsp_rmsnorm_fwd", "tsp_rmsnorm_fwd_e4m3", "tsp_rmsnorm_workspace_bytes", "tsp_rmsnorm_bwd",
    "tsp_grad_workspace_bytes", "tsp_grad_norm", "tsp_grad_clip",
]

TSP_OK, TSP_ERR_INVALID_ARG, TSP_ERR_UNSUPPORTED, TSP_ERR_CUDA, TSP_ERR_TIMEOUT = range(5)
_NAMES = {0: "TSP_OK", 1: "TSP_ERR_INVALID_ARG", 2: "TSP_ERR_UNSUPPORTED", 3: "TSP_ERR_CUDA",
          4: "TSP_ERR_TIMEOUT"}

HEADER = os.path.join(_build.ROOT, "include", "tsp.h")


class TSPError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_NAMES.get(status, status)}: {message}")
        self.status = status


class PlanInfo(ctypes.Structure):
    _fields_ = [
        ("D", ctypes.c_int), ("S", ctypes.c_int64), ("hidden", ctypes.c_int),
        ("heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("ffn", ctypes.c_int),
        ("T", ctypes.c_int64), ("C", ctypes.c_int64), ("shard_hidden", ctypes.c_int),
        ("shard_ffn", ctypes.c_int), ("shard_ffn_padded", ctypes.c_int),
        ("ffn_padded", ctypes.c_int), ("wpack_qkv", ctypes.c_size_t),
        ("wpack_o", ctypes.c_size_t), ("wpack_w13", ctypes.c_size_t),
        ("wpack_w2", ctypes.c_size_t), ("wpack_elems", ctypes.c_size_t),
        ("workspace_bytes", ctypes.c_size_t), ("bwd_workspace_bytes", ctypes.c_size_t),
        ("stat_stride", ctypes.c_int64), ("batch", ctypes.c_int), ("tokens", ctypes.c_int64),
        ("attention_group", ctypes.c_int),
    ]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


class Cost(ctypes.Structure):
    _fields_ = [
        ("devices", ctypes.c_int), ("weight_elems", ctypes.c_double),
        ("weight_inflight_elems", ctypes.c_double), ("act_elems", ctypes.c_double),
        ("act_inflight_elems", ctypes.c_double), ("comm_weight_elems", ctypes.c_double),
        ("comm_act_elems", ctypes.c_double), ("flops", ctypes.c_double),
    ]


SCHEMES = {"dp": 0, "tp": 1, "sp": 2, "tp_sp": 3, "tsp": 4}

_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_F = ctypes.c_float
_SIGS = {
    "tsp_plan": (_I, [_I, ctypes.c_int64, _I, _I, _I, ctypes.POINTER(_P)]),
    "tsp_plan_batched": (_I, [_I, ctypes.c_int64, _I, _I, _I, _I, ctypes.POINTER(_P)]),
    "tsp_plan_destroy": (None, [_P]),
    "tsp_get_plan_info": (_I, [_P, ctypes.POINTER(PlanInfo)]),
    "tsp_workspace_bytes": (ctypes.c_size_t, [_P]),
    "tsp_packed_weight_bytes": (ctypes.c_size_t, [_P]),
    "tsp_workspace_init": (_I, [_P, _P, _P]),
    "tsp_pack_weights": (_I, [_P] * 9 + [_P]),
    "tsp_shard_index": (_I, [_P, _P, _P, _P]),
    "tsp_shard": (_I, [_P, _P, _P, _P]),
    "tsp_unshard": (_I, [_P, _P, _P, _P]),
    "tsp_attention_fwd": (_I, [_P] * 6),
    "tsp_mlp_fwd": (_I, [_P] * 6),
    "tsp_mlp_fwd_noalloc": (_I, [_P] * 5),
    "tsp_layer_fwd": (_I, [_P] * 6),
    "tsp_layer_fwd_host": (_I, [_P] * 6),
    "tsp_qkv_projection": (_I, [_P, _I, _P, _P, _P, _P, _P]),
    "tsp_kv_allgather": (_I, [_P] * 5),
    "tsp_qkv_projection_gathered": (_I, [_P, _I] + [_P] * 7),
    "tsp_causal_attention_q": (_I, [_P, _I] + [_P] * 6),
    "tsp_causal_attention": (_I, [_P, _I, _P, _P, _P, _P, _P, _P]),
    "tsp_o_projection": (_I, [_P] * 8),
    "tsp_swiglu_gate_up": (_I, [_P] * 6),
    "tsp_swiglu_down": (_I, [_P] * 8),
    "tsp_device_status": (_I, [_P, _P]),
    "tsp_wait_selftest": (_I, [_P, ctypes.c_uint64, _P]),
    "tsp_last_error": (ctypes.c_char_p, []),
    "tsp_bwd_workspace_bytes": (ctypes.c_size_t, [_P]),
    "tsp_mlp_bwd": (_I, [_P] * 8),
    "tsp_unpack_weight_grads": (_I, [_P] * 10),
    "tsp_attention_bwd": (_I, [_P] * 8),
    "tsp_layer_bwd": (_I, [_P] * 8),
    "tsp_causal_attention_lse": (_I, [_P, _I] + [_P] * 7),
    "tsp_causal_attention_bwd": (_I, [_P, _I] + [_P] * 10),
    "tsp_cost_model": (_I, [_I, _I, _I, ctypes.c_int64, _I, _I, _I, ctypes.POINTER(Cost)]),
    "tsp_cost_model_batched": (_I, [_I, _I, _I, ctypes.c_int64, _I, _I, _I, _I,
                                    ctypes.POINTER(Cost)]),
    "tsp_cost_max_batch": (_I, [_I, _I, _I, ctypes.c_int64, _I, _I, _I, _I, ctypes.c_double,
                                ctypes.POINTER(ctypes.c_int64)]),
    "tsp_saved_bytes": (ctypes.c_size_t, [_P]),
    "tsp_layer_fwd_train": (_I, [_P] * 7),
    "tsp_layer_bwd_saved": (_I, [_P] * 9),
    "tsp_rank_shard_bytes": (_I, [_P, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]),
    "tsp_pack_rank_shard": (_I, [_P, _I] + [_P] * 10),
    "tsp_rank_qkv": (_I, [_P] * 7),
    "tsp_rank_kv_gather": (_I, [_P] * 5),
    "tsp_rank_attention": (_I, [_P, _I] + [_P] * 6),
    "tsp_rank_o_accumulate": (_I, [_P, _P, _P, _P, _I, _P, _P, _P, _P]),
    "tsp_rank_mlp_step": (_I, [_P] * 9),
    "tsp_packed_attention_workspace_bytes": (ctypes.c_size_t, [_L, _I, _I, _I, _I]),
    "tsp_status_init": (_I, [_P, _P]),
    "tsp_packed_attention_fwd": (_I, [_L, _I, _P, _I, _I, _I, _F] + [_P, _L] * 5 + [_P, _P]),
    "tsp_packed_attention_bwd": (_I, [_L, _I, _P, _I, _I, _I, _F] + [_P, _L] * 9 + [_P, _P]),
    "tsp_rmsnorm_fwd": (_I, [_L, _I, _P, _P, _I, _P, _F, _P, _P, _P]),
    "tsp_rmsnorm_fwd_e4m3": (_I, [_L, _I, _P, _P, _I, _P, _F, _I, _P, _P, _P, _P]),
    "tsp_rmsnorm_workspace_bytes": (ctypes.c_size_t, [_L, _I]),
    "tsp_rmsnorm_bwd": (_I, [_L, _I, _P, _I, _P, _F] + [_P] * 7),
    "tsp_grad_workspace_bytes": (ctypes.c_size_t, [_I]),
    "tsp_grad_norm": (_I, [_I] + [_P] * 6),
    "tsp_grad_clip": (_I, [_I] + [_P] * 4 + [_F] + [_P] * 3),
}


def library_path() -> str:
    return _build.LIB


def declared_functions() -> list:
    """Names of the functions include/tsp.h declares."""
    with open(HEADER) as fh:
        text = fh.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(tsp_[a-z0-9_]+)\s*\(", text)))


def load_library():
    """Load libtsp.so (built by __graft_entry__.build()); raise if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(f"libtsp.so is not built ({path}); run __graft_entry__.build() "
                           "or python -m folded_tensor_sequence_tsp_gb300.build")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def tsp_last_error() -> str:
    return load_library().tsp_last_error().decode()


def _check(status: int, name: str):
    if status != TSP_OK:
        raise TSPError(status, f"{name}: {tsp_last_error()}")


def _stream(stream):
    if stream is None:
        return _P(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, torch.cuda.Stream):
        return _P(stream.cuda_stream)
    return _P(int(stream))


def _dev(t, name, numel=None, dtype=torch.bfloat16, optional=False):
    """Pointer of a contiguous CUDA tensor of `dtype` with at least `numel` elements."""
    if t is None:
        if optional:
            return _P(None)
        raise ValueError(f"{name} is required")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")
    return _P(t.data_ptr())


def _host(t, name, numel):
    if not isinstance(t, torch.Tensor) or t.is_cuda or t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be a bfloat16 CPU tensor")
    if not t.is_contiguous() or t.numel() < numel:
        raise ValueError(f"{name} must be contiguous with {numel} elements")
    return _P(t.data_ptr())


class Plan:
    """Owns a tsp_plan_t handle."""

    def __init__(self, handle, lib):
        self._h = handle
        self._lib = lib
        info = PlanInfo()
        _check(lib.tsp_get_plan_info(handle, ctypes.byref(info)), "tsp_get_plan_info")
        self.info = info

    @property
    def handle(self):
        return self._h

    def __del__(self):
        if getattr(self, "_h", None) and self._lib is not None:
            self._lib.tsp_plan_destroy(self._h)
            self._h = None

    # shapes used by the checks below
    @property
    def act_elems(self):
        return self.info.tokens * self.info.hidden


def tsp_plan(D: int, S: int, hidden: int, heads: int, ffn: int) -> Plan:
    lib = load_library()
    h = _P()
    _check(lib.tsp_plan(D, S, hidden, heads, ffn, ctypes.byref(h)), "tsp_plan")
    return Plan(h, lib)


def tsp_plan_batched(D: int, S: int, batch: int, hidden: int, heads: int, ffn: int) -> Plan:
    """Plan for a micro-batch of `batch` sequences of S tokens (layout [D, B, S/D, H])."""
    lib = load_library()
    h = _P()
    _check(lib.tsp_plan_batched(D, S, batch, hidden, heads, ffn, ctypes.byref(h)),
           "tsp_plan_batched")
    return Plan(h, lib)


def tsp_get_plan_info(plan: Plan) -> dict:
    return plan.info.as_dict()


def tsp_workspace_bytes(plan: Plan) -> int:
    return load_library().tsp_workspace_bytes(plan.handle)


def tsp_packed_weight_bytes(plan: Plan) -> int:
    return load_library().tsp_packed_weight_bytes(plan.handle)


def _ws(plan, ws):
    return _dev(ws, "ws", tsp_workspace_bytes(plan), dtype=torch.uint8)


def _ws_status(ws):
    """Workspace of a single-step call: only its 256-byte status word is used."""
    return _dev(ws, "ws", 256, dtype=torch.uint8)


def tsp_workspace_init(plan, ws, stream=None):
    _check(load_library().tsp_workspace_init(plan.handle, _ws(plan, ws), _stream(stream)),
           "tsp_workspace_init")


def tsp_pack_weights(plan, Wq, Wk, Wv, Wo, W1, W3, W2, wpack, stream=None):
    i = plan.info
    H, F = i.hidden, i.ffn
    args = [_dev(Wq, "Wq", H * H), _dev(Wk, "Wk", H * H), _dev(Wv, "Wv", H * H),
            _dev(Wo, "Wo", H * H), _dev(W1, "W1", F * H), _dev(W3, "W3", F * H),
            _dev(W2, "W2", H * F), _dev(wpack, "wpack", i.wpack_elems)]
    _check(load_library().tsp_pack_weights(plan.handle, *args, _stream(stream)), "tsp_pack_weights")


def tsp_shard_index(plan, fwd, inv, stream=None):
    S = plan.info.tokens
    _check(load_library().tsp_shard_index(
        plan.handle, _dev(fwd, "fwd", S, torch.int32, optional=True),
        _dev(inv, "inv", S, torch.int32, optional=True), _stream(stream)), "tsp_shard_index")


def tsp_shard(plan, x, xs, stream=None):
    n = plan.act_elems
    _check(load_library().tsp_shard(plan.handle, _dev(x, "x", n), _dev(xs, "xs", n),
                                    _stream(stream)), "tsp_shard")


def tsp_unshard(plan, xs, x, stream=None):
    n = plan.act_elems
    _check(load_library().tsp_unshard(plan.handle, _dev(xs, "xs", n), _dev(x, "x", n),
                                      _stream(stream)), "tsp_unshard")


def _block(fn_name, plan, a, wpack, out, ws, stream):
    n = plan.act_elems
    fn = getattr(load_library(), fn_name)
    _check(fn(plan.handle, _dev(a, "input", n), _dev(wpack, "wpack", plan.info.wpack_elems),
              _dev(out, "out", n), _ws(plan, ws), _stream(stream)), fn_name)


def tsp_attention_fwd(plan, xs, wpack, attn, ws, stream=None):
    _block("tsp_attention_fwd", plan, xs, wpack, attn, ws, stream)


def tsp_mlp_fwd(plan, hs, wpack, mlp, ws, stream=None):
    _block("tsp_mlp_fwd", plan, hs, wpack, mlp, ws, stream)


def tsp_mlp_fwd_noalloc(plan, hs, wpack, mlp, stream=None):
    """tsp_mlp_fwd without a workspace, for callers that cannot allocate device memory
    (scratch in the library's static device buffer; see include/tsp.h)."""
    n = plan.act_elems
    _check(load_library().tsp_mlp_fwd_noalloc(
        plan.handle, _dev(hs, "hs", n), _dev(wpack, "wpack", plan.info.wpack_elems),
        _dev(mlp, "mlp", n), _stream(stream)), "tsp_mlp_fwd_noalloc")


def tsp_layer_fwd(plan, xs, wpack, out, ws, stream=None):
    _block("tsp_layer_fwd", plan, xs, wpack, out, ws, stream)


def tsp_layer_fwd_host(plan, x_host, wpack, out_host, ws, stream=None):
    n = plan.act_elems
    _check(load_library().tsp_layer_fwd_host(
        plan.handle, _host(x_host, "x_host", n), _dev(wpack, "wpack", plan.info.wpack_elems),
        _host(out_host, "out_host", n), _ws(plan, ws), _stream(stream)), "tsp_layer_fwd_host")


def tsp_qkv_projection(plan, shard, xs, wpack, qkv, ws, stream=None):
    i = plan.info
    _check(load_library().tsp_qkv_projection(
        plan.handle, int(shard), _dev(xs, "xs", plan.act_elems),
        _dev(wpack, "wpack", i.wpack_elems), _dev(qkv, "qkv", i.tokens * 3 * i.shard_hidden),
        _ws_status(ws), _stream(stream)), "tsp_qkv_projection")


def tsp_qkv_projection_gathered(plan, shard, xs, wpack, q, kn, vn, ws, stream=None):
    i = plan.info
    n = i.tokens * i.shard_hidden
    _check(load_library().tsp_qkv_projection_gathered(
        plan.handle, int(shard), _dev(xs, "xs", plan.act_elems),
        _dev(wpack, "wpack", i.wpack_elems), _dev(q, "q", n), _dev(kn, "kn", n),
        _dev(vn, "vn", n), _ws_status(ws), _stream(stream)), "tsp_qkv_projection_gathered")


def tsp_causal_attention_q(plan, shard, q, kn, vn, o, ws, stream=None):
    i = plan.info
    n = i.tokens * i.shard_hidden
    _check(load_library().tsp_causal_attention_q(
        plan.handle, int(shard), _dev(q, "q", n), _dev(kn, "kn", n), _dev(vn, "vn", n),
        _dev(o, "o", plan.act_elems), _ws_status(ws), _stream(stream)), "tsp_causal_attention_q")


def tsp_kv_allgather(plan, qkv, kn, vn, stream=None):
    i = plan.info
    n = i.tokens * i.shard_hidden
    _check(load_library().tsp_kv_allgather(
        plan.handle, _dev(qkv, "qkv", 3 * n), _dev(kn, "kn", n), _dev(vn, "vn", n),
        _stream(stream)), "tsp_kv_allgather")


def tsp_causal_attention(plan, shard, qkv, kn, vn, o, ws, stream=None):
    i = plan.info
    n = i.tokens * i.shard_hidden
    _check(load_library().tsp_causal_attention(
        plan.handle, int(shard), _dev(qkv, "qkv", 3 * n), _dev(kn, "kn", n), _dev(vn, "vn", n),
        _dev(o, "o", plan.act_elems), _ws_status(ws), _stream(stream)), "tsp_causal_attention")


def tsp_o_projection(plan, o, wpack, residual, out, ws, stream=None, out32=None):
    n = plan.act_elems
    _check(load_library().tsp_o_projection(
        plan.handle, _dev(o, "o", n), _dev(wpack, "wpack", plan.info.wpack_elems),
        _dev(residual, "residual", n, optional=True), _dev(out, "out", n),
        _dev(out32, "out32", n, torch.float32, optional=True), _ws_status(ws),
        _stream(stream)), "tsp_o_projection")


def tsp_swiglu_gate_up(plan, hs, wpack, g, ws, stream=None):
    i = plan.info
    _check(load_library().tsp_swiglu_gate_up(
        plan.handle, _dev(hs, "hs", plan.act_elems), _dev(wpack, "wpack", i.wpack_elems),
        _dev(g, "g", i.tokens * i.ffn_padded), _ws_status(ws), _stream(stream)), "tsp_swiglu_gate_up")


def tsp_swiglu_down(plan, g, wpack, residual, out, ws, stream=None, residual32=None):
    i = plan.info
    n = plan.act_elems
    _check(load_library().tsp_swiglu_down(
        plan.handle, _dev(g, "g", i.tokens * i.ffn_padded), _dev(wpack, "wpack", i.wpack_elems),
        _dev(residual, "residual", n, optional=True),
        _dev(residual32, "residual32", n, torch.float32, optional=True), _dev(out, "out", n),
        _ws_status(ws), _stream(stream)), "tsp_swiglu_down")


def tsp_device_status(ws, stream=None) -> int:
    """Synchronise the stream; return (and clear) the workspace status code."""
    return load_library().tsp_device_status(_dev(ws, "ws", 256, dtype=torch.uint8),
                                            _stream(stream))


def tsp_wait_selftest(ws, limit_ns: int, stream=None):
    _check(load_library().tsp_wait_selftest(_dev(ws, "ws", 256, dtype=torch.uint8),
                                            int(limit_ns), _stream(stream)), "tsp_wait_selftest")


# ------------------------------------------------------------------ backward

def tsp_bwd_workspace_bytes(plan: Plan) -> int:
    return load_library().tsp_bwd_workspace_bytes(plan.handle)


def _ws_bwd(plan, ws):
    return _dev(ws, "ws", tsp_bwd_workspace_bytes(plan), dtype=torch.uint8)


def tsp_mlp_bwd(plan, hs, wpack, dmlp, dhs, dwpack, ws, stream=None):
    """Backward of tsp_mlp_fwd: dhs (bf16, sharded) and the W1/W3/W2 sections of the
    packed fp32 weight gradient dwpack."""
    n = plan.act_elems
    i = plan.info
    _check(load_library().tsp_mlp_bwd(
        plan.handle, _dev(hs, "hs", n), _dev(wpack, "wpack", i.wpack_elems),
        _dev(dmlp, "dmlp", n), _dev(dhs, "dhs", n),
        _dev(dwpack, "dwpack", i.wpack_elems, torch.float32), _ws_bwd(plan, ws),
        _stream(stream)), "tsp_mlp_bwd")


def tsp_unpack_weight_grads(plan, dwpack, dWq=None, dWk=None, dWv=None, dWo=None, dW1=None,
                            dW3=None, dW2=None, stream=None):
    i = plan.info
    H, F = i.hidden, i.ffn
    f32 = torch.float32
    _check(load_library().tsp_unpack_weight_grads(
        plan.handle, _dev(dwpack, "dwpack", i.wpack_elems, f32),
        _dev(dWq, "dWq", H * H, f32, optional=True), _dev(dWk, "dWk", H * H, f32, optional=True),
        _dev(dWv, "dWv", H * H, f32, optional=True), _dev(dWo, "dWo", H * H, f32, optional=True),
        _dev(dW1, "dW1", F * H, f32, optional=True), _dev(dW3, "dW3", F * H, f32, optional=True),
        _dev(dW2, "dW2", H * F, f32, optional=True), _stream(stream)), "tsp_unpack_weight_grads")


def _bwd_block(fn_name, plan, a, wpack, g, dx, dwpack, ws, stream):
    n = plan.act_elems
    i = plan.info
    _check(getattr(load_library(), fn_name)(
        plan.handle, _dev(a, "input", n), _dev(wpack, "wpack", i.wpack_elems),
        _dev(g, "output gradient", n), _dev(dx, "input gradient", n),
        _dev(dwpack, "dwpack", i.wpack_elems, torch.float32), _ws_bwd(plan, ws),
        _stream(stream)), fn_name)


def tsp_attention_bwd(plan, xs, wpack, dattn, dxs, dwpack, ws, stream=None):
    """Backward of tsp_attention_fwd: dxs and the W_Q/W_K/W_V/W_O sections of dwpack."""
    _bwd_block("tsp_attention_bwd", plan, xs, wpack, dattn, dxs, dwpack, ws, stream)


def tsp_layer_bwd(plan, xs, wpack, dout, dxs, dwpack, ws, stream=None):
    """Backward of tsp_layer_fwd: dxs and every section of dwpack."""
    _bwd_block("tsp_layer_bwd", plan, xs, wpack, dout, dxs, dwpack, ws, stream)


def tsp_saved_bytes(plan: Plan) -> int:
    return load_library().tsp_saved_bytes(plan.handle)


def tsp_layer_fwd_train(plan, xs, wpack, out, saved, ws, stream=None):
    """tsp_layer_fwd that also keeps the attention output and row statistics in
    `saved` (a uint8 buffer of tsp_saved_bytes) for tsp_layer_bwd_saved."""
    n = plan.act_elems
    _check(load_library().tsp_layer_fwd_train(
        plan.handle, _dev(xs, "xs", n), _dev(wpack, "wpack", plan.info.wpack_elems),
        _dev(out, "out", n), _dev(saved, "saved", tsp_saved_bytes(plan), dtype=torch.uint8),
        _ws(plan, ws), _stream(stream)), "tsp_layer_fwd_train")


def tsp_layer_bwd_saved(plan, xs, wpack, saved, dout, dxs, dwpack, ws, stream=None):
    """tsp_layer_bwd using the `saved` of tsp_layer_fwd_train (no attention forward)."""
    n = plan.act_elems
    i = plan.info
    _check(load_library().tsp_layer_bwd_saved(
        plan.handle, _dev(xs, "xs", n), _dev(wpack, "wpack", i.wpack_elems),
        _dev(saved, "saved", tsp_saved_bytes(plan), dtype=torch.uint8),
        _dev(dout, "dout", n), _dev(dxs, "dxs", n),
        _dev(dwpack, "dwpack", i.wpack_elems, torch.float32), _ws_bwd(plan, ws),
        _stream(stream)), "tsp_layer_bwd_saved")


def tsp_causal_attention_lse(plan, shard, q, kn, vn, o, lse, ws, stream=None):
    i = plan.info
    n = i.tokens * i.shard_hidden
    nstat = (i.heads // i.D) * i.stat_stride
    _check(load_library().tsp_causal_attention_lse(
        plan.handle, int(shard), _dev(q, "q", n), _dev(kn, "kn", n), _dev(vn, "vn", n),
        _dev(o, "o", plan.act_elems), _dev(lse, "lse", nstat, torch.float32), _ws_status(ws),
        _stream(stream)), "tsp_causal_attention_lse")


def tsp_causal_attention_bwd(plan, shard, q, kn, vn, o, dout, lse, delta, dqkv, ws, stream=None):
    i = plan.info
    n = i.tokens * i.shard_hidden
    nstat = (i.heads // i.D) * i.stat_stride
    _check(load_library().tsp_causal_attention_bwd(
        plan.handle, int(shard), _dev(q, "q", n), _dev(kn, "kn", n), _dev(vn, "vn", n),
        _dev(o, "o", plan.act_elems), _dev(dout, "dout", plan.act_elems),
        _dev(lse, "lse", nstat, torch.float32), _dev(delta, "delta", nstat, torch.float32),
        _dev(dqkv, "dqkv", 3 * plan.act_elems), _ws_status(ws), _stream(stream)),
        "tsp_causal_attention_bwd")


def tsp_cost_model(scheme: str, D: int, S: int, hidden: int, heads: int, ffn: int, tp: int = 0) -> dict:
    """Per-device memory (elements), communication (elements received) and FLOPs of
    one layer forward under `scheme` (dp, tp, sp, tp_sp with a tp x D/tp grid, tsp)."""
    c = Cost()
    _check(load_library().tsp_cost_model(SCHEMES[scheme], D, tp, S, hidden, heads, ffn,
                                         ctypes.byref(c)), "tsp_cost_model")
    return {k: getattr(c, k) for k, _ in Cost._fields_}


def tsp_cost_model_batched(scheme: str, D: int, S: int, batch: int, hidden: int, heads: int,
                           ffn: int, tp: int = 0) -> dict:
    """tsp_cost_model for a micro-batch of `batch` sequences of S tokens."""
    c = Cost()
    _check(load_library().tsp_cost_model_batched(SCHEMES[scheme], D, tp, S, batch, hidden, heads,
                                                 ffn, ctypes.byref(c)), "tsp_cost_model_batched")
    return {k: getattr(c, k) for k, _ in Cost._fields_}


def tsp_cost_max_batch(scheme: str, D: int, S: int, hidden: int, heads: int, ffn: int,
                       layers: int, mem_bytes: float, tp: int = 0) -> int:
    """Largest micro-batch of S-token sequences whose per-device bf16 footprint for
    `layers` layers fits in mem_bytes under `scheme` (0 if one sequence does not)."""
    out = ctypes.c_int64()
    _check(load_library().tsp_cost_max_batch(SCHEMES[scheme], D, tp, S, hidden, heads, ffn,
                                             layers, float(mem_bytes), ctypes.byref(out)),
           "tsp_cost_max_batch")
    return int(out.value)


# ------------------------------------------------------------ rank-local steps

def tsp_rank_shard_bytes(plan: Plan):
    """(attention part, MLP part) bytes of one rank's weight shard."""
    a, m = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load_library().tsp_rank_shard_bytes(plan.handle, ctypes.byref(a), ctypes.byref(m)),
           "tsp_rank_shard_bytes")
    return a.value, m.value


def tsp_pack_rank_shard(plan, k, Wq, Wk, Wv, Wo, W1, W3, W2, attn_shard, mlp_shard, stream=None):
    i = plan.info
    H, F = i.hidden, i.ffn
    a, m = tsp_rank_shard_bytes(plan)
    _check(load_library().tsp_pack_rank_shard(
        plan.handle, int(k), _dev(Wq, "Wq", H * H), _dev(Wk, "Wk", H * H), _dev(Wv, "Wv", H * H),
        _dev(Wo, "Wo", H * H), _dev(W1, "W1", F * H), _dev(W3, "W3", F * H), _dev(W2, "W2", H * F),
        _dev(attn_shard, "attn_shard", a // 2), _dev(mlp_shard, "mlp_shard", m // 2),
        _stream(stream)), "tsp_pack_rank_shard")


def _rank_rows(plan):
    """Rows one rank holds: its T tokens of every sequence of the micro-batch."""
    i = plan.info
    return i.batch * i.T


def tsp_rank_qkv(plan, xs_r, attn_shard, q_r, kv_r, ws, stream=None):
    i = plan.info
    n, Hd = _rank_rows(plan), i.shard_hidden
    _check(load_library().tsp_rank_qkv(
        plan.handle, _dev(xs_r, "xs_r", n * i.hidden),
        _dev(attn_shard, "attn_shard", tsp_rank_shard_bytes(plan)[0] // 2),
        _dev(q_r, "q_r", n * Hd), _dev(kv_r, "kv_r", 2 * n * Hd), _ws_status(ws),
        _stream(stream)), "tsp_rank_qkv")


def tsp_rank_kv_gather(plan, kv_all, kn, vn, stream=None):
    i = plan.info
    n = i.tokens * i.shard_hidden
    _check(load_library().tsp_rank_kv_gather(
        plan.handle, _dev(kv_all, "kv_all", 2 * n), _dev(kn, "kn", n), _dev(vn, "vn", n),
        _stream(stream)), "tsp_rank_kv_gather")


def tsp_rank_attention(plan, r, q_r, kn, vn, o_r, ws, stream=None):
    i = plan.info
    n, nr = i.tokens * i.shard_hidden, _rank_rows(plan) * i.shard_hidden
    _check(load_library().tsp_rank_attention(
        plan.handle, int(r), _dev(q_r, "q_r", nr), _dev(kn, "kn", n), _dev(vn, "vn", n),
        _dev(o_r, "o_r", nr), _ws_status(ws), _stream(stream)), "tsp_rank_attention")


def tsp_rank_o_accumulate(plan, o_r, attn_shard, residual, acc_r, h_r, ws, stream=None):
    """acc_r = residual + o_r W_O,k^T (fp32), h_r = bf16(acc_r). residual: bf16 x_r or
    fp32 (acc_r itself)."""
    i = plan.info
    rows = _rank_rows(plan)
    n = rows * i.hidden
    f32 = residual is not None and residual.dtype == torch.float32
    _check(load_library().tsp_rank_o_accumulate(
        plan.handle, _dev(o_r, "o_r", rows * i.shard_hidden),
        _dev(attn_shard, "attn_shard", tsp_rank_shard_bytes(plan)[0] // 2),
        _dev(residual, "residual", n, torch.float32 if f32 else torch.bfloat16), int(f32),
        _dev(acc_r, "acc_r", n, torch.float32), _dev(h_r, "h_r", n), _ws_status(ws),
        _stream(stream)), "tsp_rank_o_accumulate")


def tsp_rank_mlp_step(plan, h_r, mlp_shard, residual32, acc_r, out_r, g_r, ws, stream=None):
    i = plan.info
    rows = _rank_rows(plan)
    n = rows * i.hidden
    fq = (i.shard_ffn_padded + 127) // 128 * 128
    _check(load_library().tsp_rank_mlp_step(
        plan.handle, _dev(h_r, "h_r", n),
        _dev(mlp_shard, "mlp_shard", tsp_rank_shard_bytes(plan)[1] // 2),
        _dev(residual32, "residual32", n, torch.float32), _dev(acc_r, "acc_r", n, torch.float32),
        _dev(out_r, "out_r", n), _dev(g_r, "g_r", rows * fq), _ws_status(ws), _stream(stream)),
        "tsp_rank_mlp_step")


# ------------------------------------------------------------------ around the layer
# These calls take their sizes from the tensors, and run on the tensors' device: a call
# on tensors of another device than the current one selects it for the launch.

def _same_device(tensors):
    """Index of the one CUDA device that the given tensors (None skipped) are on."""
    device = -1
    for t in tensors:
        if t is None:
            continue
        try:
            d = t.get_device()
        except AttributeError:
            d = -1
        if d < 0:
            raise ValueError("expected CUDA tensors")
        if d != device:
            if device >= 0:
                raise ValueError(f"tensors on cuda:{device} and cuda:{d}")
            device = d
    return device


def _launch(name, device, stream, *args):
    """Call `name` with the stream (default: the device's current one) as last argument."""
    fn = getattr(_lib or load_library(), name)
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device)
    else:
        raw = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    if device == torch.cuda.current_device():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status != TSP_OK:
        _check(status, name)


_STREAM_DTYPES = (torch.bfloat16, torch.float32)


def _matrix(t, name, shape=None, dtypes=(torch.bfloat16,), optional=False):
    """Pointer of a contiguous [rows, width] tensor of one of `dtypes`."""
    if t is None:
        if optional:
            return None
        raise ValueError(f"{name} is required")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    own = t.shape
    if len(own) != 2 or (shape is not None and own != shape):
        raise ValueError(f"{name} must have shape {shape or '[rows, width]'}, got {tuple(own)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _norm_args(x, weight, residual, h, *outs):
    device = _same_device((x, weight, residual, h, *outs))
    xp = _matrix(x, "x")
    shape = tuple(x.shape)
    if weight.dtype != torch.bfloat16 or weight.numel() != shape[1] or not weight.is_contiguous():
        raise ValueError(f"weight must hold {shape[1]} contiguous bfloat16 values")
    rp = _matrix(residual, "residual", shape, _STREAM_DTYPES, optional=True)
    hp = _matrix(h, "h", shape, _STREAM_DTYPES, optional=True)
    if residual is not None and (h is None or h.dtype != residual.dtype):
        raise ValueError("a residual needs an h of its type")
    if residual is None and h is not None:
        raise ValueError("h is only written with a residual")
    return device, xp, rp, hp, shape, int(residual is not None and residual.dtype == torch.float32)


def tsp_rmsnorm_fwd(x, weight, y, residual=None, h=None, eps=1e-5, stream=None):
    """h = x + residual and y = h / sqrt(mean(h^2) + eps) * weight, row by row.

    x, y: bfloat16 [rows, width]; residual and h: bfloat16 or float32 [rows, width], both or
    neither. h may be residual, y may be x."""
    device, xp, rp, hp, shape, f32 = _norm_args(x, weight, residual, h, y)
    yp = _matrix(y, "y", shape)
    _launch("tsp_rmsnorm_fwd", device, stream, shape[0], shape[1], xp, rp, f32, weight.data_ptr(),
            eps, hp, yp)


def tsp_rmsnorm_fwd_e4m3(x, weight, y, scales, residual=None, h=None, eps=1e-5, group=128,
                         stream=None):
    """tsp_rmsnorm_fwd with y in float8_e4m3fn and float32 scales: [rows, 1] with group 0,
    [rows, ceil(width / 128)] with group 128."""
    device, xp, rp, hp, shape, f32 = _norm_args(x, weight, residual, h, y, scales)
    yp = _matrix(y, "y", shape, (torch.float8_e4m3fn,))
    groups = -(-shape[1] // group) if group else 1
    sp = _matrix(scales, "scales", (shape[0], groups), (torch.float32,))
    _launch("tsp_rmsnorm_fwd_e4m3", device, stream, shape[0], shape[1], xp, rp, f32,
            weight.data_ptr(), eps, group, hp, yp, sp)


def tsp_rmsnorm_workspace_bytes(rows: int, width: int) -> int:
    return load_library().tsp_rmsnorm_workspace_bytes(rows, width)


def tsp_rmsnorm_bwd(h, weight, dy, dx, dw, ws, dh=None, dx16=None, eps=1e-5, stream=None):
    """The gradients dx of h (plus dh) and dw (float32 [width]) of the weight. h, dh and dx
    share a type, bfloat16 or float32; dx16 receives a bfloat16 copy of dx."""
    device = _same_device((h, weight, dy, dx, dw, ws, dh, dx16))
    hp = _matrix(h, "h", None, _STREAM_DTYPES)
    shape = tuple(h.shape)
    if weight.dtype != torch.bfloat16 or weight.numel() != shape[1] or not weight.is_contiguous():
        raise ValueError(f"weight must hold {shape[1]} contiguous bfloat16 values")
    if dw.dtype != torch.float32 or dw.numel() != shape[1] or not dw.is_contiguous():
        raise ValueError(f"dw must hold {shape[1]} contiguous float32 values")
    _launch("tsp_rmsnorm_bwd", device, stream, shape[0], shape[1], hp, int(h.dtype == torch.float32),
            weight.data_ptr(), eps, _matrix(dy, "dy", shape),
            _matrix(dh, "dh", shape, (h.dtype,), optional=True), _matrix(dx, "dx", shape, (h.dtype,)),
            _matrix(dx16, "dx16", shape, optional=True), dw.data_ptr(),
            _dev(ws, "ws", tsp_rmsnorm_workspace_bytes(*shape), torch.uint8))


def tsp_grad_workspace_bytes(n: int) -> int:
    return load_library().tsp_grad_workspace_bytes(n)


_GRAD_TYPES = {torch.float32: 0, torch.bfloat16: 1}


def _grad_list(grads, name):
    """(pointers, element counts, types) of the tensors as host arrays."""
    if not all([t.is_contiguous() for t in grads]):
        raise ValueError(f"{name} must be contiguous")
    types = [_GRAD_TYPES.get(t.dtype, -1) for t in grads]
    if -1 in types:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return (array.array("q", [t.data_ptr() for t in grads]), array.array("q", [t.numel() for t in grads]),
            array.array("i", types))


def _grad_args(grads, norm, ws):
    devices = {t.get_device() for t in grads}
    devices.add(_same_device((norm, ws)))
    if len(devices) != 1:
        raise ValueError("gradients, norm and ws must be on one CUDA device")
    if norm.dtype != torch.float32 or norm.numel() != 1:
        raise ValueError("norm must be one float32 value")
    return (devices.pop(), len(grads), *_grad_list(grads, "gradients"),
            _dev(ws, "ws", tsp_grad_workspace_bytes(len(grads)), torch.uint8))


def _at(values):
    """Address of a host array (the caller keeps it alive over the call)."""
    return values.buffer_info()[0] if values else None


def tsp_grad_norm(grads, norm, ws, stream=None):
    """norm (one float32 on the device) = the 2-norm over all elements of the tensors."""
    device, n, ptrs, sizes, types, wp = _grad_args(grads, norm, ws)
    _launch("tsp_grad_norm", device, stream, n, _at(ptrs), _at(sizes), _at(types), norm.data_ptr(), wp)


def tsp_grad_clip(grads, outs, max_norm, norm, ws, stream=None):
    """The norm, and outs[i] = grads[i] * min(1, max_norm / (norm + 1e-6)); outs[i] may be
    grads[i]."""
    device, n, ptrs, sizes, types, wp = _grad_args(grads, norm, ws)
    out_ptrs = ptrs
    if outs is not grads:
        out_ptrs, out_sizes, out_types = _grad_list(outs, "outs")
        if out_sizes != sizes or out_types != types or any([t.get_device() != device for t in outs]):
            raise ValueError("outs must match the gradients in number, size, type and device")
    _launch("tsp_grad_clip", device, stream, n, _at(ptrs), _at(out_ptrs), _at(sizes), _at(types), max_norm,
            norm.data_ptr(), wp)


# ------------------------------------------------------------------ packed attention

def tsp_packed_attention_workspace_bytes(tokens: int, n_seqs: int, heads: int, kv_heads: int,
                                         head_dim: int) -> int:
    return load_library().tsp_packed_attention_workspace_bytes(tokens, n_seqs, heads, kv_heads,
                                                               head_dim)


def tsp_status_init(ws, stream=None):
    """Zero the status word of a workspace that belongs to no plan."""
    _launch("tsp_status_init", _same_device((ws,)), stream, _ws_status(ws))


def _heads3(t, name, shape=None):
    """(pointer, row stride) of a bfloat16 [tokens, heads, d] tensor whose rows are contiguous."""
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    own = t.shape
    if len(own) != 3 or (shape is not None and own != shape):
        raise ValueError(f"{name} must have shape {shape or '[tokens, heads, d]'}, got {tuple(own)}")
    n, h, d = own
    row, head, one = t.stride()
    if n and h and d and (one != 1 or (h > 1 and head != d)):
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return t.data_ptr(), row if n > 1 else h * d


def _packed_args(q, k, v, starts):
    qp, ldq = _heads3(q, "q")
    kp, ldk = _heads3(k, "k")
    qs, ks = q.shape, k.shape
    tokens, heads, d = qs
    if ks[0] != tokens or ks[2] != d:
        raise ValueError(f"k has shape {tuple(ks)} beside q {tuple(qs)}")
    vp, ldv = _heads3(v, "v", ks)
    n = starts.numel() - 1
    if starts.dtype != torch.int32 or starts.dim() != 1 or n < 0 or not starts.is_contiguous():
        raise ValueError("starts must hold n_seqs + 1 contiguous int32 values")
    return (tokens, n, starts.data_ptr(), heads, ks[1], d), (qp, ldq, kp, ldk, vp, ldv), qs, ks


def _stat(t, name, heads, tokens):
    if t.dtype != torch.float32 or tuple(t.shape) != (heads, tokens):
        raise ValueError(f"{name} must be float32 [{heads}, {tokens}]")
    if tokens > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: the values of a head must be contiguous")
    if heads > 1 and t.stride(0) < tokens:
        raise ValueError(f"{name}: the rows of two heads overlap")
    return t.data_ptr(), t.stride(0) if heads > 1 else tokens


def _ws_packed(ws, sizes):
    tokens, n, _, heads, kv_heads, d = sizes
    return _dev(ws, "ws", tsp_packed_attention_workspace_bytes(tokens, n, heads, kv_heads, d),
                torch.uint8)


def tsp_packed_attention_fwd(q, k, v, starts, o, ws, lse=None, scale=None, stream=None):
    """Causal attention of packed sequences: q, o [tokens, heads, d], k, v [tokens, kv_heads, d]
    (bfloat16, rows may be strided), starts int32 [n_seqs + 1] on the device; lse float32
    [heads, tokens] receives the row statistics that the backward takes."""
    device = _same_device((q, k, v, starts, o, ws, lse))
    sizes, qkv, qs, _ = _packed_args(q, k, v, starts)
    tokens, heads, d = qs
    op, ldo = _heads3(o, "o", qs)
    lp, ldl = (None, 0) if lse is None else _stat(lse, "lse", heads, tokens)
    _launch("tsp_packed_attention_fwd", device, stream, *sizes, d ** -0.5 if scale is None else scale,
            *qkv, op, ldo, lp, ldl, _ws_packed(ws, sizes))


def tsp_packed_attention_bwd(q, k, v, starts, o, lse, dout, dq, dk, dv, ws, scale=None, stream=None):
    """Gradients of tsp_packed_attention_fwd from its o and lse and the gradient dout of o."""
    device = _same_device((q, k, v, starts, o, lse, dout, dq, dk, dv, ws))
    sizes, qkv, qs, ks = _packed_args(q, k, v, starts)
    tokens, heads, d = qs
    _launch("tsp_packed_attention_bwd", device, stream, *sizes, d ** -0.5 if scale is None else scale,
            *qkv, *_heads3(o, "o", qs), *_stat(lse, "lse", heads, tokens), *_heads3(dout, "dout", qs),
            *_heads3(dq, "dq", qs), *_heads3(dk, "dk", ks), *_heads3(dv, "dv", ks), _ws_packed(ws, sizes))
