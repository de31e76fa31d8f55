"""Refusals of the quantiser, the e4m3 products and the AdamW step, and what their objects do on the
host. No GPU: every library call below fails its checks, and what allocates or launches is replaced."""
import ctypes
import math
from types import SimpleNamespace

import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
B = tsp._binding
operators = tsp.operators


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(B.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return B.load_library()


P = lambda i: 1 << (24 + i)  # noqa: E731  distinct aligned placeholders
BAD, NO = B.TSP_ERR_INVALID_ARG, B.TSP_ERR_UNSUPPORTED


def expect(status, code, word):
    assert status == code, (status, B.tsp_last_error())
    assert word in B.tsp_last_error(), B.tsp_last_error()


def test_quantize_refusals(lib):
    def call(rows=8, width=300, x=P(0), f32=0, ldx=300, block=1, y=P(1), ldy=304, s=P(2), yt=P(3), ldyt=16, st=P(4)):
        return lib.tsp_quantize_e4m3(rows, width, x, f32, ldx, block, y, ldy, s, yt, ldyt, st, None)
    for kw, code, word in [
            (dict(rows=-1), NO, "rows"), (dict(rows=1 << 31), NO, "rows"), (dict(width=1 << 31), NO, "width"),
            (dict(width=-1), NO, "width"), (dict(block=2), NO, "blocks of"), (dict(block=0), NO, "blocks of"),
            (dict(x=None), BAD, "null"), (dict(y=None), BAD, "together"), (dict(s=None), BAD, "together"),
            (dict(yt=None), BAD, "together"), (dict(st=None), BAD, "together"),
            (dict(y=None, s=None, yt=None, st=None), BAD, "null output"),
            (dict(x=P(0) + 1), BAD, "aligned"), (dict(x=P(0) + 2, f32=1), BAD, "aligned"),
            (dict(s=P(2) + 2), BAD, "aligned"), (dict(st=P(4) + 1), BAD, "aligned"),
            (dict(ldx=299), BAD, "stride"), (dict(ldy=299), BAD, "stride"), (dict(ldyt=7), BAD, "stride"),
            (dict(ldx=(1 << 40) + 1), NO, "stride"), (dict(y=P(0)), BAD, "alias"), (dict(yt=P(1)), BAD, "alias"),
            (dict(yt=P(0)), BAD, "alias"), (dict(st=P(2)), BAD, "alias"),
            (dict(rows=(1 << 31) - 1, width=1 << 20, ldx=1 << 20, ldy=1 << 20, ldyt=1 << 31), NO, "blocks")]:
        expect(call(**kw), code, word)
    assert call(rows=0, x=None) == B.TSP_OK and call(width=0, y=None, s=None, yt=None, st=None) == B.TSP_OK


def test_matmul_refusals(lib):
    def call(m=8, n=300, k=200, a=P(0), lda=208, sa=P(1), b=P(2), ldb=208, sb=P(3), block=128, c=P(4), ldc=300, f32=0,
             acc=0, ws=P(5)):
        return lib.tsp_matmul_e4m3(m, n, k, a, lda, sa, b, ldb, sb, block, c, ldc, f32, acc, ws, None)
    for kw, code, word in [
            (dict(m=-1), NO, "m, n and k"), (dict(n=(1 << 30) + 1), NO, "m, n and k"), (dict(k=-5), NO, "m, n and k"),
            (dict(block=64), NO, "b_block"), (dict(acc=1), NO, "added"), (dict(c=None), BAD, "null"),
            (dict(c=P(4) + 1), BAD, "aligned"), (dict(c=P(4) + 2, f32=1), BAD, "aligned"), (dict(ldc=299), BAD, "stride of c"),
            (dict(a=None), BAD, "null"), (dict(b=None), BAD, "null"), (dict(sa=None), BAD, "null"), (dict(sb=None), BAD, "null"),
            (dict(a=P(0) + 8), BAD, "16 bytes"), (dict(b=P(2) + 1), BAD, "16 bytes"), (dict(lda=200), BAD, "16 bytes"),
            (dict(ldb=201), BAD, "16 bytes"), (dict(lda=192), BAD, "stride of a or b"), (dict(ldb=192), BAD, "stride of a or b"),
            (dict(sa=P(1) + 2), BAD, "aligned"), (dict(ws=None), BAD, "workspace"), (dict(ws=P(5) + 16), BAD, "256-byte"),
            (dict(c=P(0)), BAD, "alias"), (dict(c=P(2)), BAD, "alias"), (dict(c=P(1), f32=1), BAD, "alias")]:
        expect(call(**kw), code, word)
    assert call(m=0, a=None, c=None) == B.TSP_OK and call(n=0, b=None, c=None) == B.TSP_OK
    assert call(k=0, f32=1, acc=1, a=None, b=None, ws=None) == B.TSP_OK  # nothing to add
    assert tsp.tsp_matmul_e4m3_workspace_bytes() == 256


def adamw(lib, n=1, types=(0,), sizes=(300,), grad_types=None, masters=None, bits=32, params=None, grads=None, m=None,
          v=None, ms=None, vs=None, step=None, **kw):
    count = len(sizes)
    ptr = lambda x, first: (B._P * count)(*(x if x is not None else [P(0) + (first * count + i) * 65536 for i in range(count)]))  # noqa: E731
    fields = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, max_norm=1.0, t=1, seed=0)
    if step is None:
        step = B.AdamW(**{**fields, **kw})
    return lib.tsp_adamw_step(n, ptr(params, 0), (ctypes.c_int * count)(*types), None if masters is None else ptr(masters, 0),
                              ptr(grads, 1), (ctypes.c_int * count)(*(grad_types or types)), ptr(m, 2), ptr(v, 3),
                              ptr(ms, 4) if bits == 8 else None, ptr(vs, 5) if bits == 8 else None,
                              (ctypes.c_int64 * count)(*sizes), bits, ctypes.byref(step), None)


def test_adamw_refusals(lib):
    for kw, code, word in [
            (dict(beta1=1.0), BAD, "betas"), (dict(beta2=-0.1), BAD, "betas"), (dict(beta1=math.nan), BAD, "betas"),
            (dict(eps=0.0), BAD, "eps"), (dict(eps=math.inf), BAD, "eps"), (dict(eps=1e-60), BAD, "eps"), (dict(eps=1e-38), BAD, "eps"),
            (dict(lr=-1.0), BAD, "lr"), (dict(lr=math.nan), BAD, "lr"), (dict(weight_decay=-1.0), BAD, "weight_decay"),
            (dict(weight_decay=math.inf), BAD, "weight_decay"), (dict(t=0), BAD, "count from 1"),
            (dict(norm=P(9), max_norm=-1.0), BAD, "max_norm"), (dict(norm=P(9), max_norm=math.nan), BAD, "max_norm"),
            (dict(norm=P(9) + 2), BAD, "misaligned"), (dict(device_lr=P(9) + 1), BAD, "misaligned"),
            (dict(device_t=P(9) + 4), BAD, "misaligned"), (dict(bits=16), NO, "32 or 8"), (dict(n=-1), NO, "65536"),
            (dict(n=65537), NO, "65536"), (dict(sizes=[-1]), BAD, "size"), (dict(sizes=[1 << 41]), BAD, "size"),
            (dict(types=[2]), NO, "fp32 or bf16"), (dict(grad_types=[7]), NO, "fp32 or bf16"),
            (dict(masters=[P(8)]), BAD, "master"), (dict(params=[None]), BAD, "null tensor"), (dict(m=[None]), BAD, "null tensor"),
            (dict(bits=8, vs=[None]), BAD, "null tensor"), (dict(params=[P(8) + 2]), BAD, "aligned"),
            (dict(types=[1], params=[P(8) + 1]), BAD, "aligned"), (dict(types=[1], masters=[P(8) + 2]), BAD, "aligned"),
            (dict(v=[P(8) + 2]), BAD, "aligned"), (dict(bits=8, ms=[P(8) + 2]), BAD, "aligned"),
            (dict(params=[P(8)], m=[P(8)]), BAD, "overlaps"), (dict(params=[P(8)], grads=[P(8) + 400]), BAD, "overlaps"),
            (dict(m=[P(8)], v=[P(8) + 1196]), BAD, "overlaps"), (dict(bits=8, ms=[P(8)], vs=[P(8) + 8]), BAD, "overlaps"),
            (dict(n=2, sizes=[300, 300], types=[0, 0], params=[P(8), P(8)]), BAD, "overlaps")]:
        expect(adamw(lib, **kw), code, word)
    assert adamw(lib, n=0) == B.TSP_OK
    assert adamw(lib, sizes=[0]) == B.TSP_OK and adamw(lib, grads=[None]) == B.TSP_OK  # nothing to do
    assert lib.tsp_adamw_step(0, *[None] * 10, 32, None, None) == BAD


def test_the_binding_refuses_wrong_tensors():
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        tsp.tsp_quantize_e4m3(x)
    with pytest.raises(ValueError, match="CUDA"):
        tsp.tsp_adamw_step([x], [x], [x], [x], 0.1, 1)
    with pytest.raises(ValueError, match="state_bits"):
        tsp.TSPAdamW([], state_bits=16)
    with pytest.raises(ValueError, match="unsupported size"):
        tsp.TSPLinearE4M3(4, 0, 64)


# ------------------------------------------------------------------ lists of tensors on the host

def listed(tensors, **kw):
    return B.TensorList(tensors, "things", **kw)


@pytest.fixture
def on_one_device(monkeypatch):
    def get_device(t):
        if t is None:
            raise TypeError  # as the method itself does
        return 0
    monkeypatch.setattr(torch.Tensor, "get_device", get_device)


def test_lists_keep_places_sizes_and_types(on_one_device):
    a, b = torch.zeros(3, 2), torch.zeros(5, dtype=torch.bfloat16)
    full, gaps = listed([a, b]), listed([None, a, None, b])
    assert list(full.sizes) == [6, 5] and list(full.types) == [0, 1] and full.pointers[0] == a.data_ptr()
    assert list(gaps.sizes) == [0, 6, 0, 5] and list(gaps.types) == [0, 0, 0, 1]
    assert list(gaps.pointers) == [0, a.data_ptr(), 0, b.data_ptr()]
    assert listed([None, None]).device is None and listed([]).n == 0
    with pytest.raises(ValueError, match="contiguous"):
        listed([torch.zeros(4, 4)[:, :2]])
    with pytest.raises(ValueError, match="float32 or"):
        listed([torch.zeros(3, dtype=torch.float64)])


def test_lists_are_matched(on_one_device):
    weights = listed([torch.zeros(300), torch.zeros(5)])
    listed([torch.ones(300), torch.ones(5)]).like(weights, "g")
    listed([None, torch.ones(5)]).like(weights, "g")
    listed([torch.ones(3), torch.ones(1)]).like(weights, "scales", blocks=True)
    for wrong in ([torch.ones(300)], [torch.ones(5), torch.ones(300)], [None, torch.ones(0)], [None, None, None]):
        with pytest.raises(ValueError, match="match the weights"):
            listed(wrong).like(weights, "g")
    with pytest.raises(ValueError, match="match the weights"):
        listed([torch.ones(2), torch.ones(1)]).like(weights, "scales", blocks=True)


# ------------------------------------------------------------------ objects

class Fakes:
    """Constructors on the CPU: the calls that they make."""

    def __init__(self, monkeypatch):
        self.calls, self.capturing = [], False
        record = lambda name: lambda *a, **k: self.calls.append(name)  # noqa: E731

        class Device:
            def __init__(self, device):
                pass

            def __enter__(self):
                pass

            def __exit__(self, *exc):
                pass

        monkeypatch.setattr(torch.cuda, "device", Device)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)
        monkeypatch.setattr(torch.cuda, "current_stream",
                            lambda device=None: SimpleNamespace(cuda_stream=0, synchronize=record("synchronize")))
        monkeypatch.setattr(operators, "_device", lambda device: torch.device("cpu"))
        monkeypatch.setattr(operators, "tsp_status_init", record("init"))
        monkeypatch.setattr(operators, "tsp_matmul_e4m3_workspace_bytes", lambda: 256)
        monkeypatch.setattr(operators, "tsp_device_status", lambda ws, stream=None: self.calls.append(ws.numel()) or 0)
        monkeypatch.setattr(operators, "_adamw_lists", lambda *lists: lists)


def test_objects_are_ready_when_their_constructors_return(monkeypatch):
    fakes = Fakes(monkeypatch)
    layer = tsp.TSPLinearE4M3(100, 64, 32)
    assert fakes.calls == ["init", "synchronize"]
    fakes.calls.clear()
    layer.enable_backward()
    assert fakes.calls == ["init", "synchronize"]
    fakes.calls.clear()
    layer.enable_backward()  # nothing to grow
    assert fakes.calls == []
    tsp.TSPAdamW([torch.zeros(5)])
    assert fakes.calls == ["synchronize"]


def test_objects_are_not_made_in_a_capture(monkeypatch):
    fakes = Fakes(monkeypatch)
    layer = tsp.TSPLinearE4M3(100, 64, 32)
    fakes.capturing = True
    before = layer.ws
    for call in (lambda: tsp.TSPLinearE4M3(100, 64, 32), lambda: tsp.TSPAdamW([torch.zeros(5)]), layer.enable_backward):
        with pytest.raises(RuntimeError, match="before the capture"):
            call()
    assert layer.ws is before


def test_a_layers_earlier_workspace_is_kept_and_looked_at(monkeypatch):
    fakes = Fakes(monkeypatch)
    layer = tsp.TSPLinearE4M3(100, 64, 32)
    small = layer.ws.numel()
    layer.enable_backward()
    assert layer.ws.numel() > small and layer._kept[0].numel() == small
    fakes.calls.clear()
    layer.check()
    assert sorted(fakes.calls) == [small, layer.ws.numel()]


def test_a_layers_workspace_holds_its_parts():
    """Values and scales of x, of dy and of the transpose of dy, each on 256 bytes and none over another."""
    for tokens, n, k in ((0, 1, 1), (1, 1, 1), (100, 64, 33), (257, 1000, 4096)):
        layer = object.__new__(tsp.TSPLinearE4M3)
        with pytest.MonkeyPatch.context() as mp:
            Fakes(mp)
            layer.__init__(tokens, n, k)
        up16 = lambda x: -(-x // 16) * 16  # noqa: E731
        at = 256
        for (values, scales), (rows, width) in zip(layer._at, ((tokens, k), (tokens, n), (n, tokens))):
            assert values >= at and values % 256 == 0 and scales >= values + rows * up16(width) and scales % 4 == 0
            at = scales + 4 * rows * -(-width // 128)
        assert layer._sizes[1] >= at and layer._sizes[0] <= layer._at[1][0]


def test_a_master_belongs_beside_bfloat16(monkeypatch):
    Fakes(monkeypatch)
    with pytest.raises(ValueError, match="master"):
        tsp.TSPAdamW([torch.zeros(5)], masters=[torch.zeros(5)])
    with pytest.raises(ValueError, match="scales belong"):
        tsp.TSPAdamW([torch.zeros(5)]).resume(3, [torch.zeros(5)], [torch.zeros(5)], [torch.zeros(1)], [torch.zeros(1)])


@pytest.mark.parametrize("shape", [(2, 3, 64), (64,), (2, 2, 2, 16), (3, 32, 1)])
def test_an_input_in_8_bits_has_rows_of_the_layers_width(monkeypatch, shape):
    """As many values as rows of 32 have, in other rows: out is made for x's own rows, so nothing may be launched."""
    Fakes(monkeypatch)
    launched = []
    monkeypatch.setattr(operators, "_same_device", lambda tensors: 0)
    monkeypatch.setattr(operators, "_launch", lambda *args: launched.append(args))
    layer = tsp.TSPLinearE4M3(100, 48, 32)
    weight = (torch.zeros(48, 32, dtype=torch.float8_e4m3fn), torch.ones(1, 1))
    x = torch.zeros(shape, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="rows of 32"):
        layer.forward(x, weight, scales=torch.ones(x.numel() // 32, 1))
    assert not launched
    y = layer.forward(torch.zeros(2, 3, 32, dtype=torch.float8_e4m3fn), weight, scales=torch.ones(6, 1))
    assert y.shape == (2, 3, 48) and launched[0][3:6] == (6, 48, 32)


def test_adamw_check_refuses_what_the_step_does(lib):
    """The same lists with and without a stream."""
    kw = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, max_norm=1.0, t=1, seed=0)
    ptr = lambda *x: (B._P * len(x))(*x)  # noqa: E731
    ints = lambda *x: (ctypes.c_int * len(x))(*x)  # noqa: E731

    def check(g=P(1), n=1, bits=32, **change):
        return lib.tsp_adamw_check(n, ptr(P(0)), ints(0), None, ptr(g), ints(0), ptr(P(2)), ptr(P(3)), None, None,
                                   (ctypes.c_int64 * 1)(300), bits, ctypes.byref(B.AdamW(**{**kw, **change})))
    assert check() == B.TSP_OK
    expect(check(g=P(0) + 400), BAD, "overlaps")
    expect(check(bits=16), NO, "32 or 8")
    expect(check(beta1=1.0), BAD, "betas")
    expect(check(t=0), BAD, "count from 1")
    expect(check(g=P(1) + 2), BAD, "aligned")
    assert lib.tsp_adamw_check(0, *[None] * 10, 32, None) == BAD
