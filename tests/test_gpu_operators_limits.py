"""The operators around the layer at the ends of what their calls allow: offsets beyond 32
bits, buffers that are mostly empty, capacity, strides, streams used at the same time."""
import math

import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu

U = 2.0 ** -8  # half a step of bf16, relative
EPS = 1e-5


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


@pytest.fixture(autouse=True)
def free_memory():
    yield
    torch.cuda.empty_cache()


def test_attention_offsets_beyond_32_bits():
    """Sequences at the end of a buffer of 4.3e9 query elements, equal in bits to the same rows
    at the start of a small one."""
    heads, kv, d = 32, 8, 128
    rows, used = (1 << 20) + 77, 700
    n = gen(1)
    small = [n(used, h, d).bfloat16() for h in (heads, kv, kv, heads)]
    lengths = [300, 1, 0, 399]
    local = [0]
    for x in lengths:
        local.append(local[-1] + x)
    near = torch.tensor(local, dtype=torch.int32, device="cuda")
    op = tsp.TSPPackedAttention(used, 4, heads, kv, d)
    q, k, v, do = small
    o, lse = op.forward_train(q, k, v, near)
    want = (o, *op.backward(q, k, v, near, o, lse, do))
    off = rows - used
    far = near + off
    big = []
    for t in small:
        b = torch.empty((rows, *t.shape[1:]), dtype=torch.bfloat16, device="cuda")
        b[off:] = t
        big.append(b)
    Q, K, V, DO = big
    assert Q.numel() > 1 << 32
    op2 = tsp.TSPPackedAttention(rows, 4, heads, kv, d)
    O, DQ, DK, DV = torch.empty_like(Q), torch.empty_like(Q), torch.empty_like(K), torch.empty_like(V)
    LSE = torch.empty(heads, rows, device="cuda")
    op2.forward_train(Q, K, V, far, out=O, lse=LSE)
    op2.backward(Q, K, V, far, O, LSE, DO, dq=DQ, dk=DK, dv=DV)
    op2.check()
    for got, w in zip((O, DQ, DK, DV), want):
        assert torch.equal(got[off:], w)
    assert torch.equal(LSE[:, off:], lse)


def test_norm_offsets_beyond_32_bits():
    rows, width = (1 << 20) + 3, 4104
    n = gen(2)
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    assert x.numel() > 1 << 32
    tail = n(5, width).bfloat16()
    x[-5:] = tail
    w = (1 + 0.2 * n(width)).bfloat16()
    op = tsp.TSPRMSNorm(rows, width, eps=EPS)
    small = tsp.TSPRMSNorm(5, width, eps=EPS)
    y, _ = op.forward(x, w)
    assert torch.equal(y[-5:], small.forward(tail, w)[0]) and (y[:-5] == 0).all()
    del y
    y8, sc, _ = op.forward_e4m3(x, w)
    s8, ss, _ = small.forward_e4m3(tail, w)
    assert torch.equal(y8[-5:].view(torch.uint8), s8.view(torch.uint8)) and torch.equal(sc[-5:], ss)
    assert (sc[:-5] == 1).all()
    del y8, sc
    dx, dw = op.backward(x, w, x)
    sdx, sdw = small.backward(tail, w, tail)
    assert torch.equal(dx[-5:], sdx) and (dx[:-5] == 0).all()
    # zeros aside, the same five terms per column: in one chain or another
    assert ((dw - sdw).abs() <= 8 * 2.0 ** -24 * (tail.double() ** 2 / small_rms(tail)).sum(0)).all()


def small_rms(t):
    return torch.sqrt((t.double() ** 2).mean(-1, keepdim=True) + EPS)


def test_clip_offsets_beyond_32_bits():
    size = (1 << 32) + 12345
    g = torch.zeros(size, dtype=torch.bfloat16, device="cuda")
    g[-3:] = 2.0
    g[5] = 1.0
    norm = tsp.TSPGradClip(1).clip([g], 1.0)
    assert abs(norm.item() - math.sqrt(13.0)) < 1e-6
    factor = 1.0 / (math.sqrt(13.0) + 1e-6)
    assert abs(g[-1].item() - 2 * factor) <= U * 2 * factor and abs(g[5].item() - factor) <= U * factor
    assert int((g != 0).sum()) == 4


def test_clip_nothing():
    op = tsp.TSPGradClip(4)
    assert op.norm([]).item() == 0 and op.clip([], 1.0).item() == 0
    e = torch.empty(0, device="cuda")
    assert op.clip([e, e], 1.0).item() == 0


@pytest.mark.parametrize("n_seqs", [3, 400])
def test_attention_in_a_mostly_empty_buffer(n_seqs):
    """Capacity far above what is used, in tokens and in sequences; and the reverse order of
    large and small calls on one workspace."""
    heads, kv, d = 8, 2, 64
    n = gen(3)
    rows = 40000
    lengths = [7 + i % 5 for i in range(3)] + [0] * (n_seqs - 3)
    starts = [11]
    for x in lengths:
        starts.append(starts[-1] + x)
    q, do = n(rows, heads, d).bfloat16(), n(rows, heads, d).bfloat16()
    k, v = n(rows, kv, d).bfloat16(), n(rows, kv, d).bfloat16()
    far = torch.tensor(starts, dtype=torch.int32, device="cuda")
    op = tsp.TSPPackedAttention(rows, max(n_seqs, 500), heads, kv, d)
    a, b = starts[0], starts[-1]
    few = tsp.TSPPackedAttention(b, n_seqs, heads, kv, d)
    cut = [t[:b].contiguous() for t in (q, k, v, do)]
    o, lse = few.forward_train(*cut[:3], far)
    want = (o, *few.backward(*cut[:3], far, o, lse, cut[3]))
    for _ in range(2):
        O, L = op.forward_train(q, k, v, far)
        got = (O, *op.backward(q, k, v, far, O, L, do))
        op.check()
        for x, y in zip(got, want):
            assert torch.equal(x[a:b], y[a:b]) and (x[b:] == 0).all() and (x[:a] == 0).all()
        # a larger call in between
        whole = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
        op.forward(q, k, v, whole)
        # and one on the rows alone through the large workspace
        o2, _ = op.forward_train(*cut[:3], far)
        assert torch.equal(o2[a:b], o[a:b])


def test_attention_capacity_and_shapes_are_checked():
    op = tsp.TSPPackedAttention(100, 2, 4, 2, 64)
    z = lambda n, h, d=64: torch.zeros(n, h, d, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    st = torch.tensor([0, 50], dtype=torch.int32, device="cuda")
    q, k = z(50, 4), z(50, 2)
    op.forward(q, k, k, st)
    bad = [(z(101, 4), z(101, 2), z(101, 2), st), (z(50, 8), k, k, st), (q, z(50, 4), z(50, 4), st),
           (q, k, z(50, 1), st), (q, z(49, 2), k, st), (z(50, 4, 128), z(50, 2, 128), z(50, 2, 128), st),
           (q, k, k, st.long()), (q, k, k, torch.zeros(4, dtype=torch.int32, device="cuda")),
           (q, k, k, st[None]), (q.float(), k, k, st), (q, k, k, st.cpu()),
           (q.transpose(0, 1).contiguous().transpose(0, 1), k, k, st)]
    for args in bad:
        with pytest.raises((ValueError, tsp.TSPError)):
            op.forward(*args)
    with pytest.raises(tsp.TSPError):  # 8-byte aligned rows
        wide = torch.zeros(50, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")
        op.forward(wide[:, :256].unflatten(1, (4, 64)), k, k, st)
    with pytest.raises(tsp.TSPError):
        op.forward(q, k, k, st, out=q)
    for args in ((100, 2, 5, 2, 64), (100, 2, 4, 2, 96), (-1, 2, 4, 2, 64), (100, 2, 129, 1, 64)):
        with pytest.raises(tsp.TSPError):
            tsp.TSPPackedAttention(*args)


def test_norm_and_clip_arguments_are_checked():
    op = tsp.TSPRMSNorm(8, 64)
    x = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    for call in (lambda: op.forward(x.float(), w), lambda: op.forward(x, w[:32]), lambda: op.forward(x, w.float()),
                 lambda: op.forward(x, w, residual=x.half()), lambda: op.forward(x, w, residual=x[:4]),
                 lambda: op.forward(x[:, :32], w), lambda: op.forward(x, w, residual=x, h=x.float()),
                 lambda: op.forward_e4m3(x, w, group=64), lambda: op.backward(x, w, x.float()),
                 lambda: op.backward(x, w, x, dh=x.float()),
                 lambda: op.backward(torch.cat([x, x]), w, torch.cat([x, x])),
                 lambda: op.forward(torch.zeros(64, 8, dtype=torch.bfloat16, device="cuda").T, w)):
        with pytest.raises((ValueError, RuntimeError)):
            call()
    clip = tsp.TSPGradClip(2)
    f = torch.zeros(10, device="cuda")
    for call in (lambda: clip.clip([f.double()], 1.0), lambda: clip.clip([f], -1.0),
                 lambda: clip.clip([f], math.nan), lambda: clip.clip([f], 1.0, outs=[f[:5]]),
                 lambda: clip.clip([f], 1.0, outs=[f.bfloat16()]), lambda: clip.clip([f], 1.0, outs=[]),
                 lambda: clip.clip([f[::2]], 1.0), lambda: clip.clip([f.cpu()], 1.0),
                 lambda: clip.norm([f], norm=torch.zeros(2, device="cuda"))):
        with pytest.raises((ValueError, RuntimeError)):
            call()
    with pytest.raises(ValueError):  # more tensors than the workspace was made for
        clip.clip([f.clone() for _ in range(1025)], 1.0)


def test_two_streams_at_once_with_an_object_each():
    heads, kv, d, rows = 8, 2, 64, 3000
    n = gen(5)
    data, want = [], []
    lengths = ([1500, 1, 1499], [30] * 100)
    for i, ls in enumerate(lengths):
        starts = torch.tensor([0, *torch.tensor(ls).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
        q, do = n(rows, heads, d).bfloat16(), n(rows, heads, d).bfloat16()
        k, v = n(rows, kv, d).bfloat16(), n(rows, kv, d).bfloat16()
        data.append((q, k, v, starts, do))
    ops = [tsp.TSPPackedAttention(rows, 128, heads, kv, d) for _ in range(2)]
    norms = [tsp.TSPRMSNorm(rows, heads * d) for _ in range(2)]
    w = torch.ones(heads * d, dtype=torch.bfloat16, device="cuda")

    def step(i, stream=None):
        q, k, v, starts, do = data[i]
        o, lse = ops[i].forward_train(q, k, v, starts, stream=stream)
        g = ops[i].backward(q, k, v, starts, o, lse, do, stream=stream)
        y, _ = norms[i].forward(o.view(rows, -1), w, stream=stream)
        dx, dw = norms[i].backward(o.view(rows, -1), w, y, stream=stream)
        return (o, lse, *g, y, dx, dw)

    want = [step(i) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [step(i, streams[i]) for i in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    # a stream given by its handle
    got = step(0, streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want[0]))
    for op in ops:
        op.check()


def test_object_made_behind_queued_work_serves_another_stream():
    """The workspace is ready when the constructor returns, whatever its stream still has to do."""
    g = gen(3)
    q, k, v = (g(300, h, 64).bfloat16() for h in (4, 2, 2))
    starts = torch.tensor([0] + list(range(2, 301, 2)), dtype=torch.int32, device="cuda")
    want = tsp.TSPPackedAttention(300, 150, 4, 2, 64).forward(q, k, v, starts)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(20_000_000)  # about 10 ms, bounded
    op = tsp.TSPPackedAttention(300, 150, 4, 2, 64)
    op.forward(q, k, v, starts, out=out, stream=side)
    op.check(side)
    assert torch.equal(out, want)
