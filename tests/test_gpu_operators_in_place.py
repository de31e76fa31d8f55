"""The forms that write over their inputs, and strides that only some operands have, against
the plain calls: the same bits, and nothing beside the outputs touched."""
import pytest
import torch

import test_gpu_packed_attention as base

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu

# Norms: a warp's row (256, 1024), a CTA's (2048 to 16384), too wide to stage (16392, 32768);
# single elements from copies (1001, 4095, 9409 without dh) and without (9409 with dh and an
# fp32 stream, 20001). More rows than CTAs, so that rows are copied ahead of rows written.
WIDTHS = [256, 1001, 1024, 2048, 4095, 4096, 8192, 9409, 16384, 16392, 20001, 32768]
ROWS = 1300


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_backward_over_its_inputs(width, kind):
    n = gen(width)
    h, dh = n(ROWS, width).to(kind), n(ROWS, width).to(kind)
    w, dy = (1 + 0.3 * n(width)).bfloat16(), n(ROWS, width).bfloat16()
    op = tsp.TSPRMSNorm(ROWS, width)
    same = torch.equal
    for given in (None, dh):
        d16 = torch.empty_like(dy)
        dx, dw = op.backward(h, w, dy, dh=given, dx16=d16)
        assert same(d16, dx.bfloat16())
        for _ in range(3):
            y = dy.clone()  # dx16 over dy
            a, b = op.backward(h, w, y, dh=given, dx16=y)
            assert same(a, dx) and same(b, dw) and same(y, d16)
            if given is not None:
                over = given.clone()  # dx over dh, and dx16 over dy
                y = dy.clone()
                a, b = op.backward(h, w, y, dh=over, dx=over, dx16=y)
                assert a is over and same(a, dx) and same(b, dw) and same(y, d16)
            if kind == torch.bfloat16:
                y = dy.clone()  # dx over dy
                a, b = op.backward(h, w, y, dh=given, dx=y)
                assert a is y and same(a, dx) and same(b, dw)


@pytest.mark.parametrize("kind", [None, torch.bfloat16, torch.float32], ids=["none", "bf16", "fp32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_forward_over_its_inputs(width, kind):
    n = gen(width + 1)
    x = n(ROWS, width).bfloat16()
    r = None if kind is None else n(ROWS, width).to(kind)
    w = (1 + 0.3 * n(width)).bfloat16()
    op = tsp.TSPRMSNorm(ROWS, width)
    y, h = op.forward(x, w, residual=r)
    for _ in range(3):
        x2, r2 = x.clone(), None if r is None else r.clone()
        a, b = op.forward(x2, w, residual=r2, y=x2, h=r2)
        assert a is x2 and torch.equal(a, y) and (r is None or (b is r2 and torch.equal(b, h)))
    for group in (0, 128):
        y8, sc, h8 = op.forward_e4m3(x, w, residual=r, group=group)
        if r is not None:
            r2 = r.clone()
            a, s, b = op.forward_e4m3(x, w, residual=r2, group=group, h=r2)
            assert torch.equal(a.view(torch.uint8), y8.view(torch.uint8)) and torch.equal(s, sc)
            assert torch.equal(b, h8) and torch.equal(b, h)


@pytest.mark.parametrize("heads", [(4, 2, 64), (6, 2, 128), (16, 1, 64)], ids=str)
@pytest.mark.parametrize("many", [False, True], ids=["few", "many"])
def test_attention_with_strides_of_its_own_for_each_operand(heads, many):
    """o, dout and lse with gaps between their rows, each another one."""
    lengths = [130, 3, 1, 260, 8, 0, 77] + ([2, 9] * 80 if many else [])
    c = base.Case(lengths, *heads, before=3, after=6)
    op = c.op()
    o, lse = op.forward_train(c.q, c.k, c.v, c.starts)
    want = op.backward(c.q, c.k, c.v, c.starts, o, lse, c.do)
    inside = ~c.outside()

    def gaps(t, extra):
        """A copy of t [rows, heads, d] with `extra` columns of 7 behind every row."""
        whole = torch.full((t.shape[0], t.shape[1] * t.shape[2] + extra), 7.0, dtype=t.dtype, device="cuda")
        return whole, whole[:, :t.shape[1] * t.shape[2]].unflatten(1, t.shape[1:])

    whole_o, o2 = gaps(o, 8)
    o2.copy_(o)
    o2[inside] = 3
    stats = torch.full((c.heads, c.rows + 13), 7.0, device="cuda")
    lse2 = stats[:, :c.rows]
    op.forward_train(c.q, c.k, c.v, c.starts, out=o2, lse=lse2)
    op.check()
    assert torch.equal(o2[inside], o[inside]) and torch.equal(lse2[:, inside], lse[:, inside])
    assert (whole_o[:, c.heads * c.d:] == 7).all() and (stats[:, c.rows:] == 7).all()
    assert (o2[c.outside()] == 0).all() and (lse2[:, c.outside()] == 7).all()
    whole_do, do2 = gaps(c.do, 24)
    do2.copy_(c.do)
    grads = [gaps(t, e) for t, e in zip(want, (16, 40, 8))]
    op.backward(c.q, c.k, c.v, c.starts, o2, lse2, do2, *(g for _, g in grads))
    op.check()
    for (whole, got), t in zip(grads, want):
        assert torch.equal(got[inside], t[inside]) and (got[c.outside()] == 7).all()
        assert (whole[:, t.shape[1] * t.shape[2]:] == 7).all()
