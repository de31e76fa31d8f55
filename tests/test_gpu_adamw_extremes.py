"""TSPAdamW where numbers leave the ordinary range: gradients whose squares overflow, infinities and NaN. Tolerances
as in test_gpu_adamw.py, u = 2^-24."""
import math

import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BETAS, LR = (0.9, 0.95), 3e-3


def weights(kind, n, seed=1):
    """([parameter], [master] or None, dtype of its gradient)."""
    w = torch.randn(n, generator=torch.Generator().manual_seed(seed)).cuda()
    if kind == "fp32":
        return [w], None, torch.float32
    return [w.bfloat16()], [w.bfloat16().float()] if kind == "master" else None, torch.bfloat16 if kind == "bf16" else torch.float32


def gradient(n, seed):
    return torch.randn(n, generator=torch.Generator().manual_seed(seed)).cuda()


BAD = {1: 1e25, 2: math.inf, 3: math.nan, 4: -math.inf, 5: -1e30}  # block: a gradient in it; the finite ones' squares overflow


@pytest.mark.parametrize("kind", ["fp32", "bf16", "master"])
def test_a_block_of_8_bits_that_overflows_is_nan_from_then_on(kind):
    """Every weight of it, not only the element: one that stands still would not be seen. The other blocks are
    as they would have been."""
    n = 128 * 8
    p, masters, dtype = weights(kind, n)
    q, q_masters, _ = weights(kind, n)
    opt = tsp.TSPAdamW(p, masters=masters, betas=BETAS, state_bits=8)
    clean = tsp.TSPAdamW(q, masters=q_masters, betas=BETAS, state_bits=8)
    g = gradient(n, 2).to(dtype)
    opt.step([g], LR), clean.step([g], LR)
    wrong = g.clone()
    for block, value in BAD.items():
        wrong[128 * block + 7 * block] = value
    opt.step([wrong], LR), clean.step([g], LR)
    bad = torch.zeros(8, dtype=torch.bool, device="cuda")
    bad[list(BAD)] = True
    assert bool(opt.v_scales[0][bad].isnan().all()) and torch.equal(opt.v_scales[0][~bad], clean.v_scales[0][~bad])
    assert bool(opt.m_scales[0][[2, 3, 4]].isnan().all())
    for _ in range(2):
        opt.step([g], LR), clean.step([g], LR)
        for got, want in ((p, q), (masters or [], q_masters or [])):
            for a, b in zip(got, want):
                a, b = a.view(8, 128), b.view(8, 128)
                assert bool(a[bad].isnan().all()) and torch.equal(a[~bad], b[~bad])


@pytest.mark.parametrize("kind", ["fp32", "bf16", "master"])
def test_an_overflow_in_32_bits_stays_with_its_element(kind):
    n = 1000
    p, masters, dtype = weights(kind, n)
    q, q_masters, _ = weights(kind, n)
    opt = tsp.TSPAdamW(p, masters=masters, betas=BETAS)
    clean = tsp.TSPAdamW(q, masters=q_masters, betas=BETAS)
    g = gradient(n, 2).to(dtype)
    wrong = g.clone()
    wrong[5], wrong[300], wrong[999] = 1e25, math.inf, math.nan
    hit = torch.zeros(n, dtype=torch.bool, device="cuda")
    hit[[5, 300, 999]] = True
    before = p[0].clone()
    opt.step([wrong], LR), clean.step([g], LR)
    for a, b in zip(p + opt.m + opt.v, q + clean.m + clean.v):
        assert torch.equal(a[~hit], b[~hit])
    assert opt.v[0][5] == math.inf and p[0][5] == before[5]  # m / infinity
    assert bool(p[0][[300, 999]].isnan().all())
