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
    assert tsp.tsp_rmsnorm_workspace_bytes(1 << 20, 4096) == 456 * 4096 * 4
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


def test_packed_attention_refusals(lib):
    BAD, NO = B.TSP_ERR_INVALID_ARG, B.TSP_ERR_UNSUPPORTED
    base = dict(tokens=100, n=3, starts=P(0), heads=4, kv=2, d=64, scale=0.1, q=P(1), ldq=256, k=P(2),
                ldk=128, v=P(3), ldv=128, o=P(4), ldo=256, lse=P(5), ldl=100, do=P(6), lddo=256, dq=P(7),
                lddq=256, dk=P(8), lddk=128, dv=P(9), lddv=128, ws=P(10))

    def fwd(**kw):
        a = {**base, **kw}
        return lib.tsp_packed_attention_fwd(
            a["tokens"], a["n"], a["starts"], a["heads"], a["kv"], a["d"], a["scale"], a["q"], a["ldq"], a["k"],
            a["ldk"], a["v"], a["ldv"], a["o"], a["ldo"], a["lse"], a["ldl"], a["ws"], None)

    def bwd(**kw):
        a = {**base, **kw}
        return lib.tsp_packed_attention_bwd(
            a["tokens"], a["n"], a["starts"], a["heads"], a["kv"], a["d"], a["scale"], a["q"], a["ldq"], a["k"],
            a["ldk"], a["v"], a["ldv"], a["o"], a["ldo"], a["lse"], a["ldl"], a["do"], a["lddo"], a["dq"],
            a["lddq"], a["dk"], a["lddk"], a["dv"], a["lddv"], a["ws"], None)

    shared = [
        (dict(tokens=-1), NO, "tokens"), (dict(tokens=(1 << 30) + 1), NO, "tokens"),
        (dict(n=-1), NO, "sequences"), (dict(n=(1 << 20) + 1), NO, "sequences"),
        (dict(d=32), NO, "head_dim"), (dict(d=96), NO, "head_dim"), (dict(heads=5), NO, "heads"),
        (dict(heads=0), NO, "heads"), (dict(kv=0), NO, "heads"), (dict(heads=129, kv=1), NO, "heads"),
        (dict(heads=65538), NO, "heads"), (dict(heads=65536, kv=65536, tokens=1 << 30), NO, "tiles"),
        (dict(scale=0.0), BAD, "scale"), (dict(scale=-1.0), BAD, "scale"),
        (dict(scale=math.nan), BAD, "scale"), (dict(scale=math.inf), BAD, "scale"),
        (dict(starts=None), BAD, "starts"), (dict(starts=P(0) + 2), BAD, "starts"),
        (dict(q=None), BAD, "q"), (dict(k=P(2) + 8), BAD, "k"), (dict(ldq=255), BAD, "stride"),
        (dict(ldq=260), BAD, "stride"), (dict(ldk=120), BAD, "stride"), (dict(ldv=132), BAD, "stride"),
        (dict(ldo=128), BAD, "stride"), (dict(lse=P(5) + 2), BAD, "lse"), (dict(ldl=99), BAD, "lse"),
        (dict(ws=None), BAD, "workspace"), (dict(ws=P(10) + 64), BAD, "256-byte")]
    for call in (fwd, bwd):
        for kw, code, word in shared:
            expect(lib, call(**kw), code, word)
        # nothing to do: no pointer is looked at
        assert call(tokens=0, q=None, ws=None) == B.TSP_OK
        assert call(n=0, starts=None, o=None) == B.TSP_OK
    expect(lib, fwd(o=P(1)), BAD, "alias")
    expect(lib, fwd(o=P(3)), BAD, "alias")
    expect(lib, bwd(lse=None), BAD, "lse")
    for kw in (dict(dq=P(1)), dict(dk=P(2)), dict(dv=P(6)), dict(dq=P(4)), dict(dk=P(9)), dict(dv=P(7))):
        expect(lib, bwd(**kw), BAD, "alias")
    expect(lib, bwd(lddk=64), BAD, "stride")
    expect(lib, bwd(do=None), BAD, "dout")


def test_packed_attention_workspace(lib):
    size = tsp.tsp_packed_attention_workspace_bytes
    assert size(0, 0, 4, 2, 64) >= 512
    for tokens, n, heads, kv, d in [(1, 1, 1, 1, 64), (1000, 7, 32, 8, 128), (50, 4096, 130, 2, 128)]:
        tpt = 128 // (heads // kv)
        # status, counts, one item per query tile, one per key tile, Delta
        need = 512 + 16 * (tokens // tpt + n) + 16 * (tokens // 128 + n) + 4 * heads * ((tokens + 127) // 128 * 128)
        assert need <= size(tokens, n, heads, kv, d) <= need + 4 * 256
        # a workspace made for more tokens and sequences serves fewer
        assert size(tokens, n, heads, kv, d) <= size(tokens + 1, n + 1, heads, kv, d)
    assert size(100, 1, 5, 2, 64) == 0


def test_status_init_needs_a_workspace(lib):
    expect(lib, lib.tsp_status_init(None, None), B.TSP_ERR_INVALID_ARG, "workspace")
    expect(lib, lib.tsp_status_init(P(0) + 8, None), B.TSP_ERR_INVALID_ARG, "256-byte")


def test_row_statistics_whose_rows_overlap():
    one = torch.empty(1, 5)
    assert B._stat(one, "lse", 1, 5) == (one.data_ptr(), 5)
    assert B._stat(torch.empty(3, 8)[:, :5], "lse", 3, 5)[1] == 8
    for t in (one.expand(3, 5), torch.empty(9).as_strided((3, 5), (2, 1))):
        with pytest.raises(ValueError, match="overlap"):
            B._stat(t, "lse", 3, 5)
