"""Norms of rows whose sum of squares overflows fp32, as the header has them: y = 0 and h kept in
the forward, dx = dh and no share in dw in the backward; the other rows as without them."""
import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu

WIDTHS = [256, 1000, 1001, 2048, 4096, 8192, 9409, 16384, 16392, 20001]
ROWS = 40
HUGE = [0, 7, 39]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def others():
    keep = torch.ones(ROWS, dtype=torch.bool, device="cuda")
    keep[HUGE] = False
    return keep


@pytest.mark.parametrize("kind", [None, torch.bfloat16, torch.float32], ids=["none", "bf16", "fp32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_forward(width, kind):
    n = gen(width)
    x = n(ROWS, width).bfloat16()
    r = None if kind is None else n(ROWS, width).to(kind)
    w = (1 + 0.3 * n(width)).bfloat16()
    op = tsp.TSPRMSNorm(ROWS, width)
    plain, _ = op.forward(x, w, residual=r)
    x[HUGE] = 1e25
    y, h = op.forward(x, w, residual=r)
    keep = others()
    assert (y[HUGE] == 0).all() and torch.equal(y[keep], plain[keep])
    if r is not None:
        assert torch.equal(h, (x.float() + r.float()).to(kind))
    for group in (0, 128):
        y8, scales, _ = op.forward_e4m3(x, w, residual=r, group=group)
        assert (y8[HUGE].float() == 0).all() and (scales[HUGE] == 1).all()


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("width", WIDTHS)
def test_backward(width, kind):
    n = gen(width)
    h, dh = n(ROWS, width).to(kind), n(ROWS, width).to(kind)
    w, dy = (1 + 0.3 * n(width)).bfloat16(), n(ROWS, width).bfloat16()
    op = tsp.TSPRMSNorm(ROWS, width)
    keep = others()
    quiet = dy.clone()
    quiet[HUGE] = 0
    for given in (None, dh):
        plain, dw_without = op.backward(h, w, quiet, dh=given)
        spoiled = h.clone()
        spoiled[HUGE] = 1e25
        dx, dw = op.backward(spoiled, w, dy, dh=given)
        assert torch.equal(dx[keep], plain[keep]) and torch.equal(dw, dw_without)
        assert torch.equal(dx[HUGE], torch.zeros_like(dx[HUGE]) if given is None else given[HUGE])
