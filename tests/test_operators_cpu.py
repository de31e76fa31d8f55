"""Refusals of the operators around the layer, on the CPU: every call below fails its host
checks, so no pointer is followed and nothing is launched."""
import ctypes
import math

import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
B = tsp._binding


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(B.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return B.load_library()


P = lambda i: 1 << (24 + i)  # noqa: E731  distinct aligned placeholders


def expect(lib, status, code, word):
    assert status == code, (status, B.tsp_last_error())
    assert word in B.tsp_last_error(), B.tsp_last_error()


def test_rmsnorm_forward_refusals(lib):
    def call(rows=4, width=64, x=P(0), r=None, f32=0, w=P(1), eps=1e-5, h=None, y=P(2)):
        return lib.tsp_rmsnorm_fwd(rows, width, x, r, f32, w, eps, h, y, None)
    BAD, NO = B.TSP_ERR_INVALID_ARG, B.TSP_ERR_UNSUPPORTED
    for kw, code, word in [
            (dict(rows=-1), NO, "rows"), (dict(rows=1 << 31), NO, "rows"),
            (dict(width=0), NO, "width"), (dict(width=32769), NO, "width"),
            (dict(eps=0.0), BAD, "eps"), (dict(eps=-1.0), BAD, "eps"),
            (dict(eps=math.nan), BAD, "eps"), (dict(eps=math.inf), BAD, "eps"),
            (dict(x=None), BAD, "null"), (dict(w=None), BAD, "null"), (dict(y=None), BAD, "null"),
            (dict(x=P(0) + 1), BAD, "aligned"), (dict(r=P(3) + 2, h=P(4), f32=1), BAD, "aligned"),
            (dict(r=P(3)), BAD, "residual"), (dict(h=P(3)), BAD, "residual"),
            (dict(r=P(3), h=P(0)), BAD, "alias"), (dict(r=P(3), h=P(3), y=P(3)), BAD, "alias")]:
        expect(lib, call(**kw), code, word)
    assert call(rows=0) == B.TSP_OK
    for group in (1, 64, 256, -128):
        expect(lib, lib.tsp_rmsnorm_fwd_e4m3(4, 64, P(0), None, 0, P(1), 1e-5, group, None, P(2), P(3),
                                             None), NO, "group")
    expect(lib, lib.tsp_rmsnorm_fwd_e4m3(4, 64, P(0), None, 0, P(1), 1e-5, 0, None, P(2), None, None),
           BAD, "null")
    expect(lib, lib.tsp_rmsnorm_fwd_e4m3(4, 64, P(0), None, 0, P(1), 1e-5, 0, None, P(0), P(3), None),
           BAD, "alias")


def test_rmsnorm_backward_refusals(lib):
    def call(rows=4, width=64, h=P(0), f32=0, w=P(1), eps=1e-5, dy=P(2), dh=None, dx=P(3), dx16=None,
             dw=P(4), ws=P(5)):
        return lib.tsp_rmsnorm_bwd(rows, width, h, f32, w, eps, dy, dh, dx, dx16, dw, ws, None)
    BAD, NO = B.TSP_ERR_INVALID_ARG, B.TSP_ERR_UNSUPPORTED
    for kw, code, word in [
            (dict(rows=-1), NO, "rows"), (dict(width=40000), NO, "width"), (dict(eps=0.0), BAD, "eps"),
            (dict(h=None), BAD, "null"), (dict(dy=None), BAD, "null"), (dict(dx=None), BAD, "null"),
            (dict(dw=None), BAD, "null"), (dict(ws=None), BAD, "workspace"),
            (dict(ws=P(5) + 16), BAD, "256-byte"), (dict(h=P(0) + 2, f32=1), BAD, "aligned"),
            (dict(dx=P(0)), BAD, "alias"), (dict(dx16=P(3)), BAD, "alias"),
            (dict(dx16=P(0)), BAD, "alias"), (dict(f32=1, dx=P(2)), BAD, "alias")]:
        expect(lib, call(**kw), code, word)
    assert tsp.tsp_rmsnorm_workspace_bytes(0, 64) == 256
    assert tsp.tsp_rmsnorm_workspace_bytes(3, 100) == 1280
    assert tsp.tsp_rmsnorm_workspace_bytes(1 << 20, 4096) == 304 * 4096 * 4
    assert tsp.tsp_rmsnorm_workspace_bytes(4, 0) == 0


def test_grad_refusals(lib):
    def call(ptrs, outs=None, sizes=None, types=None, max_norm=1.0, norm=P(6), ws=P(7), n=None):
        n = len(ptrs) if n is None else n
        arr = lambda t, v: (t * len(v))(*v)  # noqa: E731
        outs = ptrs if outs is None else outs
        return lib.tsp_grad_clip(n, arr(B._P, ptrs), arr(B._P, outs),
                                 arr(ctypes.c_int64, sizes or [100] * len(ptrs)),
                                 arr(ctypes.c_int, types or [0] * len(ptrs)), max_norm, norm, ws, None)
    BAD, NO = B.TSP_ERR_INVALID_ARG, B.TSP_ERR_UNSUPPORTED
    for args, kw, code, word in [
            ([P(0)], dict(max_norm=-1.0), BAD, "max_norm"), ([P(0)], dict(max_norm=math.nan), BAD, "max_norm"),
            ([P(0)], dict(norm=None), BAD, "norm"), ([P(0)], dict(ws=None), BAD, "workspace"),
            ([P(0)], dict(types=[2]), NO, "fp32 or bf16"), ([P(0)], dict(sizes=[-1]), BAD, "size"),
            ([P(0)], dict(sizes=[1 << 41]), BAD, "size"), ([None], {}, BAD, "null"),
            ([P(0) + 2], {}, BAD, "aligned"), ([P(0) + 1], dict(types=[1]), BAD, "aligned"),
            ([P(0)], dict(n=-1), NO, "65536"), ([P(0)], dict(n=65537), NO, "65536"),
            ([P(0), P(0)], {}, BAD, "overlaps"), ([P(0), P(0) + 396], {}, BAD, "overlaps"),
            ([P(0)], dict(outs=[P(0) + 4]), BAD, "overlaps"),
            ([P(0), P(1)], dict(outs=[P(1), P(0)]), BAD, "overlaps"),
            ([P(0), P(1)], dict(outs=[P(2), P(2) + 200]), BAD, "overlaps")]:
        expect(lib, call(args, **kw), code, word)
    assert tsp.tsp_grad_workspace_bytes(0) == tsp.tsp_grad_workspace_bytes(1024) == 608 * 8
    assert tsp.tsp_grad_workspace_bytes(1025) == 2 * 608 * 8
    assert tsp.tsp_grad_workspace_bytes(-1) == tsp.tsp_grad_workspace_bytes(65537) == 0


def test_binding_refuses_wrong_tensors(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        tsp.tsp_rmsnorm_fwd(x, x[0], x)
    with pytest.raises(ValueError, match="CUDA"):
        tsp.tsp_grad_norm([x], x, x)
