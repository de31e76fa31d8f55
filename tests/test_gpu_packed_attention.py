"""Packed attention with grouped heads on the GPU, against the formula in float64.

Tolerances, from the arithmetic (u = 2^-8, half a step of bf16 relative to the value):
* o_i = sum_j p_ij v_j / l_i. Each P is rounded once to bf16 (u of its term, so at most
  u sum_j p_ij |v_j| / l_i), l and the products are fp32, and o is rounded once (u |o|).
  fp32 work: the scores' sums of d products (d 2^-24 of sum |q||k|, times scale log2(e),
  enters the exponent), the exponential (2^-22) and sums of up to L terms; bounded below by
  F = (2^-20 + 2^-18) of the same magnitude for the sizes here.
* lse: the exponent's error as above plus 2^-22, absolute, and half an fp32 step.
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
