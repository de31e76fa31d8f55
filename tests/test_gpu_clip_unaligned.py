"""The gradient norm of tensors that do not start on 16 bytes, where rounding shows: every
thread's first square is 1 and the others lie just below half a step of 1, so a sum that takes
them one after the other keeps none.

Bound. A thread's squares (64 to a chunk, two more at the ends of an unaligned one) lie in four
chains of at most 17, each term rounded once as it is added (2^-24 of the chain's sum, all terms
positive), and two levels join the chains: 19 2^-24 of the sum. The rest is fp64. The root halves
it, and the norm is rounded once: 11 2^-24."""
import math

import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu

BOUND = 11 * 2.0 ** -24
SMALL = 2.0 ** -12 * (255 / 256)  # exact in bf16; its square is 0.992 2^-24


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("offset", [0, 1, 2, 3, 4, 5, 7, 8])
@pytest.mark.parametrize("n", [1, 2, 7, 300, 16383, 16384, 16385, 50001])
def test_norm_of_a_slice(dtype, offset, n):
    flat = torch.full((n + 16,), 1e30, device="cuda", dtype=dtype)  # nothing beside the slice counts
    g = flat[offset:offset + n]
    g.fill_(SMALL)
    for first in range(0, n, 16384):  # the first element of every thread, in each chunk
        g[first:first + 256] = 1.0
    want = math.sqrt(float((g.double() ** 2).sum()))
    op = tsp.TSPGradClip(1)
    norm = op.norm([g]).item()
    assert abs(norm - want) <= BOUND * want, ((norm / want - 1) * 2 ** 24, "units of 2^-24")
    keep = flat.clone()
    op.clip([g], 0.5 * want)
    # the factor's error is the norm's and one rounding; then the product's and the type's
    factor = 0.5 * want / (want + 1e-6)
    got = flat[offset:offset + n].double()
    err = (got - keep[offset:offset + n].double() * factor).abs()
    half = torch.finfo(dtype).eps / 2
    assert (err <= (half + BOUND + 3 * 2.0 ** -24) * keep[offset:offset + n].double() * factor).all()
    assert torch.equal(flat[:offset], keep[:offset]) and torch.equal(flat[offset + n:], keep[offset + n:])


@pytest.mark.parametrize("offset", [0, 1, 3])
def test_whole_range_of_a_slice(offset):
    """Squares that overflow or vanish in fp32, and values that are not finite, at both ends."""
    op = tsp.TSPGradClip(1)
    for size in (1e30, 1e-40):
        flat = torch.zeros(20011, device="cuda")
        g = flat[offset:offset + 20000]
        g.fill_(size)
        want = math.sqrt(float((g.double() ** 2).sum()))
        assert abs(op.norm([g]).item() - want) <= BOUND * want + 2.0 ** -149
    for where in (0, 1, 2, 3, 19996, 19999):
        flat = torch.zeros(20011, device="cuda")
        g = flat[offset:offset + 20000]
        g[where] = math.inf
        assert math.isinf(op.norm([g]).item())
        g[where] = math.nan
        assert math.isnan(op.norm([g]).item())
