"""The AdamW step on every pair of a weight's and a gradient's type, and the call on lists beside the object.
Tolerances and helpers of test_gpu_adamw.py."""
import pytest
import torch

from test_gpu_adamw import BETAS, DECAY, EPS, LR, SIZES, check_step, make, snapshot

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [0, 1, 4])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "master"])
def test_a_gradient_of_the_other_type(kind, bits, offset):
    kinds = [kind] * len(SIZES)
    opt, params, masters, grads = make(kinds, SIZES, bits, 3, offset)

    def place(g):
        g = g.float() if kind == "bf16" else g.bfloat16()
        buf = torch.zeros(g.numel() + offset, dtype=g.dtype, device="cuda")[offset:]
        return buf.copy_(g)

    grads = [place(g) for g in grads]
    before = snapshot(opt, params, masters)
    opt.step(grads, LR)
    check_step(opt, params, masters, grads, kinds, before, 41)


@pytest.mark.parametrize("bits", [32, 8])
def test_the_call_on_lists_is_the_objects(bits):
    kinds, sizes = ["fp32", "master", "bf16", "master"], [500, 4097, 130, 64]
    a, b = make(kinds, sizes, bits, 12), make(kinds, sizes, bits, 12)
    norm = torch.tensor(2.0, device="cuda")
    for t in (41, 42):
        a[0].step([a[3][0], None, *a[3][2:]], LR, norm=norm, max_norm=1.0)
        o = b[0]
        args = (b[1], [b[3][0], None, *b[3][2:]], o.m, o.v, LR, t)
        kw = dict(masters=b[2], m_scales=o.m_scales, v_scales=o.v_scales, betas=BETAS, eps=EPS, weight_decay=DECAY, norm=norm,
                  max_norm=1.0, seed=o.seed)
        tsp.tsp_adamw_check(*args, **kw)
        tsp.tsp_adamw_step(*args, **kw)
    for x, y in zip(a[1] + a[2][1:2] + a[0].m + a[0].v, b[1] + b[2][1:2] + b[0].m + b[0].v):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    with pytest.raises(tsp.TSPError, match="overlaps"):
        tsp.tsp_adamw_check(b[1], b[1], o.m, o.v, LR, 43, **kw)
