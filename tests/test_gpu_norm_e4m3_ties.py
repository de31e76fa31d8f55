"""The 8-bit norm's scales and values, bit for bit. Rows are built so that y is known exactly in
fp32: a quarter of the columns holds 2 and the others 0, so the mean of the squares is 1, eps =
1e-30 vanishes beside it, rstd is 1 and y = 2 w. Then scale = max|y| / 448 and y / scale are
each one fp32 division, rounded to nearest, and the value is the nearest e4m3 of that quotient,
to even at a tie. A reciprocal in place of either division misses ties."""
import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu

EPS = 1e-30


def expected(y, group):
    rows, width = y.shape
    g = group or width
    groups = -(-width // g)
    padded = torch.nn.functional.pad(y, (0, groups * g - width)).view(rows, groups, g)
    top = padded.abs().amax(-1)
    scales = torch.where(top > 0, (top / 448).clamp_min(2.0 ** -126), torch.ones_like(top))
    return scales, (padded / scales[..., None]).view(rows, -1)[:, :width].to(torch.float8_e4m3fn)


def rows_of(width, kind, weight):
    """x, residual and the exact y for the weight."""
    rows = 5
    x = torch.zeros(rows, width, dtype=torch.bfloat16)
    for i in range(rows):
        x[i, (4 * torch.arange(width // 4) + i) % width] = 2.0
    r = None if kind is None else torch.zeros(rows, width, dtype=kind)
    return x, r, x.float() * weight.float()


# a warp's row (256, 512, 1024), a CTA's (2048, 8192), too wide to stage (16384 + 128), single
# elements (132, 4100)
@pytest.mark.parametrize("width", [128, 132, 256, 512, 1024, 2048, 4100, 8192, 16512])
@pytest.mark.parametrize("group", [0, 128])
def test_scales_and_values_bit_for_bit(width, group):
    g = torch.Generator().manual_seed(width)
    op = tsp.TSPRMSNorm(5, width, eps=EPS)
    # quotients that are ties between two e4m3 values: 448 v / top = m with m halfway
    ties = torch.tensor([25.0, 27.0, 29.0, 31.0, 17.0, 19.0, 21.0, 23.0])
    for trial in range(12):
        # the last ones: scales that are small, clamped, and large
        size = {8: 2.0 ** -70, 9: 2.0 ** -115, 10: 2.0 ** -128, 11: 2.0 ** 100}.get(trial, 1.0)
        w = (torch.randn(width, generator=g) * size).bfloat16()
        if trial in (1, 3, 5, 7):
            k = trial
            w = (ties[torch.randint(0, 8, (width,), generator=g)] * (k / 64)).bfloat16()
            # the top of every group, in each row's own quarter of the columns
            for c in range(0, width, 128):
                w[c:c + 4] = 7.0 * k
        for kind in (None, torch.bfloat16, torch.float32):
            x, r, y = rows_of(width, kind, w)
            want_s, want_y = expected(y, group)
            y8, scales, _ = op.forward_e4m3(x.cuda(), w.cuda(), residual=None if r is None else r.cuda(), group=group)
            assert torch.equal(scales.cpu(), want_s), (trial, kind)
            assert torch.equal(y8.cpu().view(torch.uint8), want_y.view(torch.uint8)), (trial, kind)


@pytest.mark.parametrize("width", [128, 132, 2048, 16512])
@pytest.mark.parametrize("group", [0, 128])
def test_an_infinite_value_leaves_zeros_beside_it(width, group):
    """An infinite y has an infinite scale: a finite value's quotient is 0, its own NaN."""
    w = torch.ones(width).bfloat16()
    w[4] = float("inf")
    x = torch.zeros(1, width, dtype=torch.bfloat16)
    x[0, ::4] = 2.0
    x[0, 2::4] = 2.0 ** -70  # (its square vanishes beside the others)
    y8, scales, _ = tsp.TSPRMSNorm(1, width, eps=EPS).forward_e4m3(x.cuda(), w.cuda(), group=group)
    assert torch.isinf(scales[0, 0])
    got = y8.cpu().float()[0]
    assert torch.isnan(got[4])
    got[4] = 0
    assert (got[:128] == 0).all()
