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


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-8, 1e-15, 1e-25, 1e-30])
def test_roots_of_second_moments_below_the_normal_numbers(eps, bits):
    """v = (1 - beta2) g^2 from 2^-116 down to 300 steps of 2^-149: its root counts beside a small eps, as the rule has it.
    g^2 and v are rounded to steps of 2^-149, half of one each; the root takes half of v's relative error."""
    n = 4000
    b1, b2 = BETAS
    sign = gradient(n, 3).sign()
    g = (10 ** torch.linspace(-20.5, -17, n, dtype=torch.float64)).float().cuda() * sign
    p = torch.zeros(n, device="cuda")
    tsp_opt = tsp.TSPAdamW([p], betas=BETAS, eps=eps, state_bits=bits)
    tsp_opt.step([g], LR)
    g = g.double()
    v = (1 - b2) * g * g
    want = -LR * g / ((v / (1 - b2)).sqrt() + eps)  # m is corrected to g
    error = 20 * U + 0.5 * 2.0 ** -150 * (1 + (1 - b2)) / v
    assert bool(((p.double() - want).abs() <= error * want.abs()).all()), float(((p.double() - want).abs() / want.abs() / error).max())


def test_steps_whose_parts_are_below_the_normal_numbers():
    """g^2 is 0 in fp32, so the step is rate * m / eps; rate * m, which takes half a step of 2^-149, is not lost."""
    n, eps = 1000, 2e-37
    g = torch.linspace(1e-37, 9e-37, n, device="cuda")
    p = torch.zeros(n, device="cuda")
    tsp.TSPAdamW([p], betas=BETAS, eps=eps).step([g], LR)
    want = -LR * g.double() / eps
    assert bool(((p.double() - want).abs() <= 20 * U * want.abs() + 2.0 ** -149 / eps).all())
