"""Packed attention over sequences of a few tokens, which single warps take, beside ones that
tiles take: against the formula in float64 with the bounds of the packed attention's own tests
(the same roundings, but that the forward keeps P in fp32), found in registers and from the
list, and with values that are not finite in masked places."""
import pytest
import torch

import test_gpu_packed_attention as base

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu

HEADS = [(1, 1, 64), (3, 3, 128), (8, 2, 128), (10, 2, 64), (16, 2, 64), (32, 1, 128), (33, 1, 64), (14, 2, 128)]


def run(c):
    op = c.op()
    o = torch.full((c.rows, c.heads, c.d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.heads, c.rows), 7.0, device="cuda")
    op.forward_train(c.q, c.k, c.v, c.starts, out=o, lse=lse)
    grads = op.backward(c.q, c.k, c.v, c.starts, o, lse, c.do)
    op.check()
    return (o, lse, *grads)


@pytest.mark.parametrize("heads", HEADS, ids=lambda h: "%dof%dx%d" % h)
@pytest.mark.parametrize("n", [1, 2, 9, 40, 129, 700])
def test_each_short_length(heads, n):
    lengths = [(i * 7 + 8) % 10 for i in range(n)]
    c = base.Case(lengths, *heads, before=3, after=5)
    o, lse, *grads = run(c)
    base.check_forward(c, o, lse, f"{n}")
    base.check_backward(c, grads, f"{n}")
    out = c.outside()
    assert (o[out] == 7).all() and (lse[:, out] == 7).all()


@pytest.mark.parametrize("heads", [(8, 2, 128), (6, 2, 64)], ids=str)
def test_short_beside_long_keep_their_bits(heads):
    """Sequences of 1 to 9 tokens alone, behind a long one, and among more than 128."""
    lengths = [1, 8, 2, 7, 9, 3, 6, 4, 5]
    total = sum(lengths)
    c = base.Case([600] + lengths + [0] * 60 + [3] * 90, *heads)
    want = run(c)
    base.check_forward(c, want[0], want[1], "mixed")
    base.check_backward(c, want[2:], "mixed")
    alone = base.Case(lengths, *heads, fused=False)
    s = slice(600, 600 + total)
    alone.q, alone.k, alone.v, alone.do = (t[s].contiguous() for t in (c.q, c.k, c.v, c.do))
    for x, y in zip(run(alone), want):
        assert torch.equal(x, y[:, s] if y.dtype == torch.float32 else y[s])


@pytest.mark.parametrize("heads", [(8, 2, 128), (5, 1, 64)], ids=str)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")], ids=str)
def test_later_tokens_and_neighbours_that_are_not_finite(heads, value):
    """K and V of the last token of every second sequence: the forward's rows before it and all
    of the other sequences keep their bits. (Within its own sequence the gradient of an earlier
    query is, as the formula has it, a sum with 0 times that key, which is not 0.)"""
    lengths = [6, 5, 1, 4, 3, 2]
    c = base.Case(lengths, *heads, fused=False)
    clean = run(c)
    bad = torch.zeros(c.rows, dtype=torch.bool, device="cuda")
    own = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    for i in range(0, len(lengths), 2):
        bad[c.starts_host[i + 1] - 1] = True
        own[c.starts_host[i]:c.starts_host[i + 1]] = False
    c.k = c.k.clone()
    c.v = c.v.clone()
    c.k[bad] = value
    c.v[bad] = value
    o, lse, dq, dk, dv = run(c)
    assert torch.equal(o[~bad], clean[0][~bad])
    assert torch.equal(lse[:, ~bad], clean[1][:, ~bad])
    for got, want in zip((dq, dk, dv), clean[2:]):
        assert torch.equal(got[own], want[own])


def test_starts_out_of_order_leave_short_sequences_alone():
    c = base.Case([3, 4, 5], 4, 2, 64, after=20)
    op = c.op()
    starts = torch.tensor([0, 3, 2, 5], dtype=torch.int32, device="cuda")
    o = torch.full((c.rows, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    op.forward(c.q, c.k, c.v, starts, out=o)
    with pytest.raises(tsp.TSPError):
        op.check()
    assert (o == 7).all()
