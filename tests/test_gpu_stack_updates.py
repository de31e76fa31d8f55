"""TSPStack's AdamW steps: what a refused step leaves."""
import pytest
import torch

import gpu_util as gu
import tsp_inputs

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu
D, S, H, HEADS, F = 2, 256, 256, 4, 320


def normal(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


def made(**kw):
    """A stack of two layers with updates, and gradients of all its weights."""
    weights = []
    for i in range(2):
        b = tsp_inputs.layer_inputs(tsp_inputs.LayerConfig("t", D, S, H, HEADS, F, 21 + i))
        w = {k: gu.dev(b[k]) for k in ("Wq", "Wk", "Wv", "Wo", "W1", "W3", "W2")}
        w["attn_norm"], w["mlp_norm"] = ((1 + 0.2 * normal(H, seed=i)).bfloat16() for _ in range(2))
        weights.append(w)
    stack = tsp.TSPStack(D, S, H, HEADS, F, weights, (1 + 0.2 * normal(H, seed=7)).bfloat16())
    stack.enable_updates(**kw)
    return stack, [0.1 * normal(p.numel(), seed=30 + i) for i, p in enumerate(stack.wpack + stack.norms)]


def everything(stack):
    out = stack.wpack + stack.norms + [m for ms in stack.masters for m in ms]
    for o in stack.optimizers:
        out = out + o.m + o.v + (o.m_scales or []) + (o.v_scales or [])
    return [x.clone().view(torch.uint8) for x in out]


@pytest.mark.parametrize("bits", [32, 8])
def test_a_refused_step_leaves_everything(bits):
    stack, grads = made(state_bits=bits)
    stack.step(grads, 1e-3)
    before = everything(stack)
    for wrong in (grads[:-1], grads[:-1] + [grads[-1][:-1]], grads + grads[:1], grads[:-1] + [stack.masters[1][-1]],
                  grads[:-1] + [stack.norms[-1]]):
        with pytest.raises((ValueError, tsp.TSPError)):
            stack.step(wrong, 1e-3)
    with pytest.raises(tsp.TSPError):
        stack.step(grads, 1e-3, max_norm=-1.0)
    assert all(torch.equal(a, b) for a, b in zip(before, everything(stack))) and [o.t for o in stack.optimizers] == [1, 1]
    stack.step(grads, 1e-3)
    assert not any(torch.equal(a, b) for a, b in zip(before[:9], everything(stack))) and [o.t for o in stack.optimizers] == [2, 2]


def test_updates_enabled_again_go_on_from_the_masters():
    stack, grads = made()
    for _ in range(3):
        stack.step(grads, 1e-4)
    masters = [m.clone() for ms in stack.masters for m in ms]
    assert not all(torch.equal(p.float(), m) for p, m in zip(stack.wpack + stack.norms, masters))
    stack.norms[0].fill_(0.75)
    stack.enable_updates(state_bits=8)
    written = masters[len(stack.wpack)]
    written[written.bfloat16() != 0.75] = 0.75  # what the others hold beyond the weight stays
    assert all(torch.equal(a, b) for a, b in zip(masters, [m for ms in stack.masters for m in ms]))
    stack.step(grads, 1e-4)
    assert [o.t for o in stack.optimizers] == [1, 1]
    assert all(torch.equal(p, m.bfloat16()) for p, m in zip(stack.wpack + stack.norms, [m for ms in stack.masters for m in ms]))
