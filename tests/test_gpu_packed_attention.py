"""Packed attention with grouped heads on the GPU, against the formula in float64.

Tolerances, from the arithmetic (u = 2^-8, half a step of bf16 relative to the value):
* o_i = sum_j p_ij v_j / l_i. Each P is rounded once to bf16 (u of its term, so at most
  u sum_j p_ij |v_j| / l_i), l and the products are fp32, and o is rounded once (u |o|).
  fp32 work: the scores' sums of d products (d 2^-24 of sum |q||k|, times scale log2(e),
  enters the exponent), the exponential (2^-22) and sums of up to L terms; bounded below by
  F = (2^-20 + 2^-18) of the same magnitude for the sizes here.
* lse: the exponent's error as above plus 2^-22, absolute, and half an fp32 step.
* The backward forms P again from lse (relative error E = 4 times the exponent's bound, plus
  2^-20 for the exponential and lse's own rounding) and rounds P and dS to bf16 once each:
    dv_j: u |dv| + sum_i (u + E_i) P_ij |dO_i|
    dS_ij: u |dS| + P_ij (delta_i + d 2^-24 sum_c |dO||v|) + E_i P_ij (|dP_ij| + |Delta_i|)
  where delta_i bounds Delta's error, which comes from the rounded o of the forward:
  sum_c |dO_ic| times o's bound. dq and dk: u of the value, and scale times dS's bound
  against |k| and |q|. fp32 sums over up to L terms add F of the sums of magnitudes.
"""
import math

import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu

U = 2.0 ** -8
F = 2.0 ** -20 + 2.0 ** -18
HEADS = [(1, 1, 64), (4, 4, 64), (6, 2, 64), (7, 1, 128), (8, 2, 128), (10, 2, 64), (32, 1, 64),
         (128, 1, 64), (130, 2, 128), (3, 3, 128)]
LENGTHS = {
    "one token": [1],
    "ones": [1] * 9,
    "two": [2, 1],
    "short": [5, 0, 1, 17, 64, 3],
    "tile edges": [127, 128, 129, 1, 255, 256, 257],
    "empty ends": [0, 0, 130, 0],
    "several tiles": [700, 1, 385],
    "many": [(i * 7) % 23 for i in range(150)],
}


class Case:
    def __init__(self, lengths, heads, kv, d, seed=0, before=0, after=0, fused=True, magnitude=1.0):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed + 1000 * heads + d)
        n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.lengths, self.heads, self.kv, self.d = lengths, heads, kv, d
        starts = [before]
        for x in lengths:
            starts.append(starts[-1] + x)
        self.starts_host = starts
        self.rows = starts[-1] + after
        self.starts = torch.tensor(starts, dtype=torch.int32, device="cuda")
        if fused:
            qkv = (n(self.rows, (heads + 2 * kv) * d) * magnitude).bfloat16()
            self.q = qkv[:, :heads * d].unflatten(1, (heads, d))
            self.k = qkv[:, heads * d:(heads + kv) * d].unflatten(1, (kv, d))
            self.v = qkv[:, (heads + kv) * d:].unflatten(1, (kv, d))
        else:
            self.q = (n(self.rows, heads, d) * magnitude).bfloat16()
            self.k = (n(self.rows, kv, d) * magnitude).bfloat16()
            self.v = (n(self.rows, kv, d) * magnitude).bfloat16()
        self.do = n(self.rows, heads, d).bfloat16()
        self.scale = d ** -0.5

    def op(self, **kw):
        return tsp.TSPPackedAttention(max(self.rows, 1), len(self.lengths), self.heads, self.kv, self.d, **kw)

    def sequences(self):
        """(rows, q, k, v, do) of every sequence that has tokens, in float64, [heads][L][d], key
        heads repeated for their group."""
        G = self.heads // self.kv
        for a, b in zip(self.starts_host, self.starts_host[1:]):
            if b > a:
                f = lambda t, r: t[a:b].double().transpose(0, 1).repeat_interleave(r, 0)  # noqa: E731
                yield slice(a, b), f(self.q, 1), f(self.k, G), f(self.v, G), f(self.do, 1)

    def outside(self):
        """Mask of the rows that belong to no sequence."""
        m = torch.ones(self.rows, dtype=torch.bool, device="cuda")
        m[self.starts_host[0]:self.starts_host[-1]] = False
        return m


def softmax_parts(q, k, scale):
    L = q.shape[1]
    s = (q @ k.transpose(1, 2)) * scale
    hidden = torch.ones(L, L, dtype=torch.bool, device="cuda").triu(1)
    s = s.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(s, -1)
    # the exponent's error bound per row: fp32 sums of d products
    mag = (q.abs() @ k.abs().transpose(1, 2)).masked_fill(hidden, 0).amax(-1) * scale
    return torch.exp(s - lse[..., None]), lse / math.log(2.0), q.shape[2] * 2.0 ** -24 * mag * 2


def within(got, want, bound, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), f"{what}: non-finite"
    worst = ((got - want).abs() - bound).max().item()
    assert worst <= 0, f"{what}: {worst:.3e} over the bound"


def check_forward(c, o, lse, what):
    for rows, q, k, v, _ in c.sequences():
        p, elog, err = softmax_parts(q, k, c.scale)
        mag = p @ v.abs()
        within(o[rows].transpose(0, 1), p @ v,
               U * (p @ v).abs() + (U + F + 4 * err[..., None]) * mag, f"{what} o {rows}")
        if lse is not None:
            within(lse[:, rows], elog, 2 * err * math.log2(math.e) + 2.0 ** -21 + 2.0 ** -23 * elog.abs(),
                   f"{what} lse {rows}")


def exact_backward(c, q, k, v, do):
    """Exact dq, dk, dv of one sequence (per query head) and their bounds."""
    p, _, err = softmax_parts(q, k, c.scale)
    E = (4 * err + 2.0 ** -20)[..., None]
    o = p @ v
    obound = U * o.abs() + (U + F + 4 * err[..., None]) * (p @ v.abs())
    dp = do @ v.transpose(1, 2)
    delta = (do * o).sum(-1, keepdim=True)
    ds = p * (dp - delta)
    dmag = do.abs() @ v.abs().transpose(1, 2)
    edelta = (do.abs() * obound).sum(-1, keepdim=True) + c.d * 2.0 ** -24 * (do * o).abs().sum(-1, keepdim=True)
    eds = (U + F) * ds.abs() + p * (edelta + c.d * 2.0 ** -24 * dmag) + E * p * (dp.abs() + delta.abs())
    G = c.heads // c.kv
    group = lambda t: t.unflatten(0, (c.kv, G)).sum(1)  # noqa: E731
    dq, bq = c.scale * (ds @ k), c.scale * (eds @ k.abs())
    dk, bk = group(c.scale * (ds.transpose(1, 2) @ q)), group(c.scale * (eds.transpose(1, 2) @ q.abs()))
    dv, bv = group(p.transpose(1, 2) @ do), group(((U + F + E) * p).transpose(1, 2) @ do.abs())
    return [(x, b + (U + F) * x.abs() + 2.0 ** -133) for x, b in ((dq, bq), (dk, bk), (dv, bv))]


def check_backward(c, grads, what):
    for rows, q, k, v, do in c.sequences():
        for name, got, (want, bound) in zip(("dq", "dk", "dv"), grads, exact_backward(c, q, k, v, do)):
            within(got[rows].transpose(0, 1), want, bound, f"{what} {name} {rows}")


@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%dof%dx%d" % h)
def test_forward(lengths, heads):
    c = Case(LENGTHS[lengths], *heads, before=3, after=5)
    op = c.op()
    o = torch.full((c.rows, c.heads, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.heads, c.rows), 7.0, device="cuda")
    op.forward_train(c.q, c.k, c.v, c.starts, out=o, lse=lse)
    op.check()
    check_forward(c, o, lse, lengths)
    # rows of no sequence are left as they were
    assert (o[c.outside()] == 7).all() and (lse[:, c.outside()] == 7).all()
    o2 = op.forward(c.q, c.k, c.v, c.starts)
    assert (o2[c.outside()] == 0).all()
    inside = ~c.outside()
    assert torch.equal(o[inside], o2[inside])


@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 2, 128)], ids=str)
def test_long_sequence_and_sharp_scores(heads):
    """Several thousand keys; scores large enough that the running maximum moves."""
    c = Case([3001, 40], *heads, fused=False, magnitude=3.0)
    op = c.op()
    o, lse = op.forward_train(c.q, c.k, c.v, c.starts)
    op.check()
    check_forward(c, o, lse, "sharp")


def test_scale_argument():
    c = Case([200, 33], 4, 2, 64)
    c.scale = 0.31
    o, lse = c.op(scale=0.31).forward_train(c.q, c.k, c.v, c.starts)
    check_forward(c, o, lse, "scale")


@pytest.mark.parametrize("heads", [(6, 2, 64), (4, 4, 128)], ids=str)
def test_a_sequence_does_not_see_its_neighbours(heads):
    """The same bits alone and packed, beside NaN, infinities and rows of no sequence."""
    lengths = [130, 70, 257, 1]
    c = Case(lengths, *heads, before=2, after=90)
    op = c.op()
    o, lse = op.forward_train(c.q, c.k, c.v, c.starts)
    for bad in (math.nan, math.inf, -math.inf):
        for s in (1, 2):
            q, k, v = c.q.clone(), c.k.clone(), c.v.clone()
            a, b = c.starts_host[s], c.starts_host[s + 1]
            for t in (q, k, v):
                t[a:b] = bad
                t[c.outside()] = bad
            o2, lse2 = op.forward_train(q, k, v, c.starts)
            keep = torch.ones(c.rows, dtype=torch.bool, device="cuda")
            keep[a:b] = False
            assert torch.equal(o2[keep], o[keep]) and torch.equal(lse2[:, keep], lse[:, keep])
            assert torch.isnan(o2[a:b]).all()
    for a, b in zip(c.starts_host, c.starts_host[1:]):
        alone = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        o1, lse1 = op.forward_train(c.q[a:b].contiguous(), c.k[a:b].contiguous(), c.v[a:b].contiguous(), alone)
        assert torch.equal(o1, o[a:b]) and torch.equal(lse1, lse[:, a:b])


def test_more_than_a_thousand_sequences():
    c = Case([1 + (i * 11) % 7 for i in range(2000)], 8, 2, 64)
    op = c.op()
    o = op.forward(c.q, c.k, c.v, c.starts)
    op.check()
    G = c.heads // c.kv
    # every sequence at once: a dense mask per block of 500 sequences
    for s0 in range(0, 2000, 500):
        a, b = c.starts_host[s0], c.starts_host[s0 + 500]
        ids = torch.repeat_interleave(torch.arange(500, device="cuda"),
                                      torch.tensor(c.lengths[s0:s0 + 500], device="cuda"))
        f = lambda t, r: t[a:b].double().transpose(0, 1).repeat_interleave(r, 0)  # noqa: E731
        q, k, v = f(c.q, 1), f(c.k, G), f(c.v, G)
        sc = (q @ k.transpose(1, 2)) * c.scale
        hidden = (ids[:, None] != ids[None, :]) | torch.ones(b - a, b - a, dtype=torch.bool, device="cuda").triu(1)
        p = torch.softmax(sc.masked_fill(hidden, -math.inf), -1)
        within(o[a:b].transpose(0, 1), p @ v, U * (p @ v).abs() + (U + 4 * F) * (p @ v.abs()), f"block {s0}")


@pytest.mark.parametrize("starts", [[0, 5, 3, 10], [-1, 5], [0, 11], [4, 2], [0, 1 << 30]], ids=str)
def test_bad_starts_are_reported_and_write_nothing(starts):
    c = Case([10], 4, 2, 64)
    op = tsp.TSPPackedAttention(10, 4, 4, 2, 64)
    o = torch.full_like(c.do, 3)
    bad = torch.tensor(starts, dtype=torch.int32, device="cuda")
    op.forward(c.q, c.k, c.v, bad, out=o)
    with pytest.raises(tsp.TSPError) as e:
        op.check()
    assert e.value.status == tsp.TSP_ERR_INVALID_ARG and "starts" in str(e.value)
    assert (o == 3).all()
    op.forward(c.q, c.k, c.v, c.starts, out=o)
    op.check()
    check_forward(c, o, None, "after")


@pytest.mark.parametrize("where", [0, 150, 398])
def test_bad_starts_among_many_sequences(where):
    """The same where the kernels take their items from a list."""
    c = Case([5] * 399, 4, 2, 64)
    op = c.op()
    o, lse = op.forward_train(c.q, c.k, c.v, c.starts)
    bad = c.starts.clone()
    bad[where] = -1 if where == 0 else bad[where + 1] + 3
    out = torch.full_like(c.do, 3)
    grads = [torch.full_like(t, 3) for t in (c.do, c.k.contiguous(), c.v.contiguous())]
    op.forward(c.q, c.k, c.v, bad, out=out)
    with pytest.raises(tsp.TSPError):
        op.check()
    op.backward(c.q, c.k, c.v, bad, o, lse, c.do, *grads)
    with pytest.raises(tsp.TSPError):
        op.check()
    assert (out == 3).all() and all((g == 3).all() for g in grads)
    again = op.forward(c.q, c.k, c.v, c.starts)
    op.check()
    assert torch.equal(again, o)


def test_no_tokens_and_no_sequences():
    op = tsp.TSPPackedAttention(16, 4, 4, 2, 64)
    e = lambda n, h: torch.empty(n, h, 64, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert op.forward(e(0, 4), e(0, 2), e(0, 2), none).shape == (0, 4, 64)
    assert (op.forward(e(16, 4), e(16, 2), e(16, 2), none) == 0).all()
    assert (op.forward(e(16, 4), e(16, 2), e(16, 2), torch.full((4,), 7, dtype=torch.int32, device="cuda")) == 0).all()
    op.check()


def test_replay_with_other_lengths_on_another_stream():
    """starts is data: a captured call replays with new lengths and new inputs."""
    a, b = Case([100, 20, 300], 8, 2, 64, seed=1), Case([7, 380, 33], 8, 2, 64, seed=2)
    op = a.op()
    want = [op.forward_train(c.q, c.k, c.v, c.starts) for c in (a, b)]
    q, k, v, starts = a.q.clone(), a.k.clone(), a.v.clone(), a.starts.clone()
    o, lse = torch.zeros_like(want[0][0]), torch.zeros_like(want[0][1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            op.forward_train(q, k, v, starts, out=o, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    for c, (wo, wl) in ((b, want[1]), (a, want[0])):
        for x, y in ((q, c.q), (k, c.k), (v, c.v), (starts, c.starts)):
            x.copy_(y)
        graph.replay()
        assert torch.equal(o, wo) and torch.equal(lse, wl)
    op.check()


# ------------------------------------------------------------------ backward

@pytest.mark.parametrize("lengths", list(LENGTHS))
@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%dof%dx%d" % h)
def test_backward(lengths, heads):
    c = Case(LENGTHS[lengths], *heads, before=3, after=5)
    op = c.op()
    o, lse = op.forward_train(c.q, c.k, c.v, c.starts)
    # the three gradients as column ranges of one buffer
    full = torch.full((c.rows, (c.heads + 2 * c.kv) * c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    a, b = c.heads * c.d, (c.heads + c.kv) * c.d
    grads = (full[:, :a].unflatten(1, (c.heads, c.d)), full[:, a:b].unflatten(1, (c.kv, c.d)),
             full[:, b:].unflatten(1, (c.kv, c.d)))
    op.backward(c.q, c.k, c.v, c.starts, o, lse, c.do, *grads)
    op.check()
    check_backward(c, grads, lengths)
    assert (full[c.outside()] == 7).all()
    again = op.backward(c.q, c.k, c.v, c.starts, o, lse, c.do)
    op.check()
    inside = ~c.outside()
    for x, y in zip(grads, again):
        assert torch.equal(x[inside], y[inside]) and (y[c.outside()] == 0).all()


@pytest.mark.parametrize("heads", [(4, 2, 64), (8, 2, 128), (6, 1, 128)], ids=str)
def test_backward_long_sequence_and_sharp_scores(heads):
    c = Case([2001, 40], *heads, fused=False, magnitude=2.0)
    op = c.op()
    o, lse = op.forward_train(c.q, c.k, c.v, c.starts)
    grads = op.backward(c.q, c.k, c.v, c.starts, o, lse, c.do)
    op.check()
    check_backward(c, grads, "sharp")


@pytest.mark.parametrize("heads", [(6, 2, 64), (4, 4, 128), (7, 1, 64)], ids=str)
def test_backward_of_a_sequence_does_not_see_its_neighbours(heads):
    lengths = [130, 70, 257, 1, 30]
    c = Case(lengths, *heads, before=2, after=90)
    op = c.op()
    o, lse = op.forward_train(c.q, c.k, c.v, c.starts)
    grads = op.backward(c.q, c.k, c.v, c.starts, o, lse, c.do)
    for bad in (math.nan, math.inf):
        for s in (1, 2):
            a, b = c.starts_host[s], c.starts_host[s + 1]
            keep = torch.ones(c.rows, dtype=torch.bool, device="cuda")
            keep[a:b] = False
            spoiled = [t.clone() for t in (c.q, c.k, c.v, o, lse.T, c.do)]
            for t in spoiled:
                t[~keep] = bad
                t[c.outside()] = bad
            q, k, v, o2, lse2, do = spoiled
            got = op.backward(q, k, v, c.starts, o2, lse2.T.contiguous(), do)
            for x, y in zip(got, grads):
                assert torch.equal(x[keep], y[keep])
                assert torch.isnan(x[a:b]).any()
    for a, b in zip(c.starts_host, c.starts_host[1:]):
        alone = torch.tensor([0, b - a], dtype=torch.int32, device="cuda")
        f = lambda t: t[a:b].contiguous()  # noqa: E731
        got = op.backward(f(c.q), f(c.k), f(c.v), alone, f(o), lse[:, a:b].contiguous(), f(c.do))
        for x, y in zip(got, grads):
            assert torch.equal(x, y[a:b])


def test_backward_matches_differences():
    """The gradients along random directions against central differences of the formula."""
    c = Case([9, 4], 6, 2, 64, fused=False)
    op = c.op()
    o, lse = op.forward_train(c.q, c.k, c.v, c.starts)
    grads = op.backward(c.q, c.k, c.v, c.starts, o, lse, c.do)
    step = 1e-5
    for rows, q, k, v, do in c.sequences():
        G = c.heads // c.kv
        shared = lambda t: t[::G]  # noqa: E731  undo the repetition
        bounds = [b for _, b in exact_backward(c, q, k, v, do)]

        def loss(qq, kk, vv):
            p, _, _ = softmax_parts(qq, kk.repeat_interleave(G, 0), c.scale)
            return (do * (p @ vv.repeat_interleave(G, 0))).sum()

        args = [q, shared(k), shared(v)]
        for i in range(3):
            for seed in range(4):
                g = torch.Generator(device="cuda")
                g.manual_seed(seed)
                way = torch.randn(args[i].shape, generator=g, device="cuda", dtype=torch.float64)
                up, down = list(args), list(args)
                up[i], down[i] = args[i] + step * way, args[i] - step * way
                want = ((loss(*up) - loss(*down)) / (2 * step)).item()
                got = (grads[i][rows].transpose(0, 1).double() * way).sum().item()
                # the differences' own error is of order step^2 and 1e-16 / step
                assert abs(got - want) <= (bounds[i] * way.abs()).sum().item() + 1e-6


def test_backward_in_a_graph_beside_a_live_eager_graph():
    """Captured forward and backward replay with other lengths while eager results live."""
    a, b = Case([100, 20, 300], 8, 2, 64, seed=1), Case([7, 380, 33], 8, 2, 64, seed=2)
    op = a.op()

    def step(q, k, v, starts, do):
        o, lse = op.forward_train(q, k, v, starts)
        return (o, lse, *op.backward(q, k, v, starts, o, lse, do))

    want = [step(c.q, c.k, c.v, c.starts, c.do) for c in (a, b)]
    buf = [t.clone() for t in (a.q, a.k, a.v, a.starts, a.do)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step(*buf)
    torch.cuda.current_stream().wait_stream(side)
    for c, w in ((b, want[1]), (a, want[0])):
        for x, y in zip(buf, (c.q, c.k, c.v, c.starts, c.do)):
            x.copy_(y)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(out, w))
    op.check()


def test_backward_bad_starts_write_nothing():
    c = Case([10], 4, 2, 64)
    op = tsp.TSPPackedAttention(10, 4, 4, 2, 64)
    o, lse = op.forward_train(c.q, c.k, c.v, c.starts)
    grads = [torch.full_like(t, 3) for t in (c.q.contiguous(), c.k.contiguous(), c.v.contiguous())]
    op.backward(c.q, c.k, c.v, torch.tensor([0, 9, 4], dtype=torch.int32, device="cuda"), o, lse, c.do, *grads)
    with pytest.raises(tsp.TSPError):
        op.check()
    assert all((g == 3).all() for g in grads)
