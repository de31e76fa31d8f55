"""How far a NaN or an infinity in one token's row reaches inside its own sequence of the
packed attention. A pair above the diagonal has P = 0 and dS = 0 but stands in a tile's product
all the same, where 0 times a value that is not finite is not 0. With TPT = 128 // G tokens to
a query tile, which begins at a multiple of TPT, and key tiles of 128 positions:

* the query tile from t0 on takes keys below ceil((t0 + TPT) / 128) 128, so a key row reaches
  o and dq of at most that - 1 - t0 positions before it;
* the key tile from k0 on takes query tiles from floor(k0 / TPT) TPT on, so a query's row reaches
  dk and dv of at most k0 + 127 minus that positions after it.

Both are at most R = 127 where TPT divides 128, and 126 + TPT otherwise. Rows further away, and
the row statistics, keep their bits. (Where causality has it, the results are not finite.)"""
import math

import pytest
import torch

import test_gpu_packed_attention as base

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu

HEADS = [(4, 4, 64), (6, 2, 64), (5, 1, 128), (14, 2, 128), (65, 1, 64)]
LENGTH = 700
PLACES = [0, 125, 128, 255, 300, 511, 640, 699]


def reach(G):
    tpt = 128 // G
    return 127 if 128 % tpt == 0 else 126 + tpt


@pytest.fixture(scope="module", params=HEADS, ids=lambda h: "%dof%dx%d" % h)
def case(request):
    c = base.Case([5, LENGTH, 40], *request.param, fused=False)
    op = c.op()
    o, lse = op.forward_train(c.q, c.k, c.v, c.starts)
    grads = op.backward(c.q, c.k, c.v, c.starts, o, lse, c.do)
    op.check()
    return c, op, o, lse, grads


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf], ids=str)
@pytest.mark.parametrize("at", PLACES)
def test_a_key_row(case, at, value):
    """k and v of one token: rows of o and dq before its reach, and every earlier lse."""
    c, op, o, lse, grads = case
    start, end = c.starts_host[1], c.starts_host[2]
    row = start + at
    k, v = c.k.clone(), c.v.clone()
    k[row] = value
    v[row] = value
    o2, lse2 = op.forward_train(c.q, k, v, c.starts)
    dq, dk, dv = op.backward(c.q, k, v, c.starts, o2, lse2, c.do)
    op.check()
    far = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    far[max(start, row - reach(c.heads // c.kv)):end] = False
    assert torch.equal(o2[far], o[far]) and torch.equal(dq[far], grads[0][far])
    before = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    before[row:end] = False
    assert torch.equal(lse2[:, before], lse[:, before])
    other = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    other[start:end] = False
    assert torch.equal(dk[other], grads[1][other]) and torch.equal(dv[other], grads[2][other])
    assert not torch.isfinite(o2[row:end]).all(-1).any()  # every later query sees it


@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf], ids=str)
@pytest.mark.parametrize("which", ["q", "o", "do"])
@pytest.mark.parametrize("at", PLACES)
def test_a_query_row(case, at, which, value):
    """q, o or dout of one token in the backward: dq of every other token, and dk and dv of the
    tokens behind its reach."""
    c, op, o, lse, grads = case
    start, end = c.starts_host[1], c.starts_host[2]
    row = start + at
    args = {"q": c.q.clone(), "o": o.clone(), "do": c.do.clone()}
    args[which][row] = value
    dq, dk, dv = op.backward(args["q"], c.k, c.v, c.starts, args["o"], lse, args["do"])
    op.check()
    others = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    others[row] = False
    assert torch.equal(dq[others], grads[0][others])
    far = torch.ones(c.rows, dtype=torch.bool, device="cuda")
    far[start:min(end, row + reach(c.heads // c.kv) + 1)] = False
    assert torch.equal(dk[far], grads[1][far]) and torch.equal(dv[far], grads[2][far])
    if which == "do":
        assert not torch.isfinite(dv[start:row + 1]).all(-1).any()  # every earlier key is seen by it


def test_the_formula_of_the_reach_holds_for_every_group(case):
    """The tile geometry of the docstring, counted out."""
    for G in range(1, 129):
        tpt = 128 // G
        before = max(-(-(t0 + tpt) // 128) * 128 - 1 - t0 for t0 in range(0, 128 * tpt, tpt))
        after = max(k0 + 127 - k0 // tpt * tpt for k0 in range(0, 128 * tpt, 128))
        assert max(before, after) <= reach(G)
        assert (128 % tpt == 0) == (max(before, after) == 127)
