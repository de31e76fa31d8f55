"""The operators together, as a training step in 8 bits uses them, and TSPStack's steps.

Tolerances: the layers' products are held in test_gpu_matmul_e4m3.py and the update in
test_gpu_adamw.py; here each call's result is compared with what 64 bits make of the results of the calls
before it, rounded as those calls say."""
import math

import pytest
import torch

import gpu_util as gu
import tsp_inputs

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24
BETAS, LR, DECAY = (0.9, 0.95), 1e-2, 0.1


def wide(x, scales, block):
    s = scales.double().repeat_interleave(128, 1)[:, :x.shape[1]]
    if block == 128:
        s = s.repeat_interleave(128, 0)[:x.shape[0]]
    return x.float().double() * s


def quantised(x):
    q = torch.empty(x.shape, dtype=E4M3, device="cuda")
    s = torch.empty(x.shape[0], -(-x.shape[1] // 128), device="cuda")
    tsp.tsp_quantize_e4m3(x, q, s)
    return wide(q, s, 1)


def near(got, want, size, terms):
    """fp32 sums of `terms` products, as in test_gpu_matmul_e4m3.py, and one rounding to bf16."""
    tol = (131 + terms / 128) * U * size
    if got.dtype == torch.bfloat16:
        tol = tol + (want.abs() + tol) * 2.0 ** -8
    assert bool(((got.double() - want).abs() <= tol).all())


def normal(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


@pytest.mark.parametrize("bits", [32, 8])
def test_two_layers_learn_for_some_steps(bits):
    """norm -> 8-bit layer -> 8-bit layer, backward, global norm, update of fp32 masters, weights quantised
    again: twice, so that the second step runs on what the first has left."""
    tokens, width, inner = 200, 256, 384
    masters = [0.05 * normal(inner, width, seed=1), 0.05 * normal(width, inner, seed=2)]
    params = [m.bfloat16() for m in masters]
    norm_w = torch.ones(width, dtype=torch.bfloat16, device="cuda")
    layers = [tsp.TSPLinearE4M3(tokens, inner, width), tsp.TSPLinearE4M3(tokens, width, inner)]
    norm, clip = tsp.TSPRMSNorm(tokens, width), tsp.TSPGradClip(2)
    opt = tsp.TSPAdamW(params, masters=masters, betas=BETAS, weight_decay=DECAY, state_bits=bits)
    x, dy = normal(tokens, width, seed=3).bfloat16(), normal(tokens, width, seed=4).bfloat16()
    for step in (1, 2):
        weights = [l.quantize_weight(m) for l, m in zip(layers, masters)]
        h, _ = norm.forward(x, norm_w)
        a, saved_a = layers[0].forward_train(h, weights[0])
        y, saved_y = layers[1].forward_train(a, weights[1])
        da, dw1 = layers[1].backward(saved_y, dy, weights[1])
        dx, dw0 = layers[0].backward(saved_a, da, weights[0])
        grads = [dw0, dw1]
        total = clip.norm(grads)
        before = [m.double() for m in masters]
        m_before = [wide_state(opt, i, "m") for i in range(2)]
        v_before = [wide_state(opt, i, "v") for i in range(2)]
        opt.step(grads, LR, norm=total, max_norm=1.0)

        w64 = [wide(w.values, w.scales, 128) for w in weights]
        a64, y64 = quantised(h), quantised(a)
        near(a, a64 @ w64[0].t(), a64.abs() @ w64[0].abs().t(), width)
        near(y, y64 @ w64[1].t(), y64.abs() @ w64[1].abs().t(), inner)
        g = quantised(dy)
        near(da, g @ w64[1], g.abs() @ w64[1].abs(), width)
        gt, at = quantised(dy.t().contiguous()), quantised(a.t().contiguous())
        near(dw1, gt @ at.t(), gt.abs() @ at.abs().t(), tokens)
        g = quantised(da)
        near(dx, g @ w64[0], g.abs() @ w64[0].abs(), inner)
        want = math.sqrt(sum(float(w.double().square().sum()) for w in grads))
        assert abs(float(total) - want) <= 1e-6 * want
        factor = min(1.0, 1.0 / (float(total) + 1e-6))
        for i in range(2):
            gi = grads[i].double() * factor
            m1 = BETAS[0] * m_before[i] + (1 - BETAS[0]) * gi
            v1 = BETAS[1] * v_before[i] + (1 - BETAS[1]) * gi * gi
            move = m1 / (1 - BETAS[0] ** step) / ((v1 / (1 - BETAS[1] ** step)).sqrt() + 1e-8)
            p1 = before[i] - LR * (DECAY * before[i] + move)
            # the update's parts are off by 24 u each; with beta1 m and (1 - beta1) g of either sign, m by 4 u of both
            parts = (BETAS[0] * m_before[i]).abs() + ((1 - BETAS[0]) * gi).abs()
            size = LR * (DECAY * before[i].abs() + (move * parts / m1.abs().clamp_min(1e-300)).abs())
            assert bool(((masters[i].double() - p1).abs() <= U * p1.abs() + 24 * U * size + 1e-12).all())
            assert torch.equal(params[i], masters[i].bfloat16())
    for layer in layers:
        layer.check()


def wide_state(opt, i, name):
    x = getattr(opt, name)[i].view(-1)
    if opt.state_bits == 8:
        s = getattr(opt, name + "_scales")[i]
        x = x.float().double() * s.double().repeat_interleave(128)[:x.numel()]
    return x.double().view(opt.params[i].shape)


def test_a_whole_step_replays_from_a_graph():
    """Quantised weights, forward, backward, norm and update in one graph, with t and lr on the device: the masters
    after three replays are those of three eager steps."""
    tokens, n, k = 130, 200, 256
    x, dy = normal(tokens, k, seed=3).bfloat16(), normal(tokens, n, seed=4).bfloat16()
    results = []
    for captured in (False, True):
        master = 0.05 * normal(n, k, seed=1)
        param = master.bfloat16()
        layer, clip = tsp.TSPLinearE4M3(tokens, n, k), tsp.TSPGradClip(1)
        layer.enable_backward()
        opt = tsp.TSPAdamW([param], masters=[master], betas=BETAS, state_bits=8)
        lr, t = torch.tensor(LR, device="cuda"), torch.ones((), dtype=torch.int64, device="cuda")

        def step():
            w = layer.quantize_weight(master)
            y, saved = layer.forward_train(x, w)
            _, dw = layer.backward(saved, dy, w)
            opt.step([dw], lr, norm=clip.norm([dw]), max_norm=1.0, t=t)
            t.add_(1)

        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for _ in range(3):
            graph.replay() if captured else step()
        torch.cuda.synchronize()
        layer.check()
        results.append((master, param, opt.m[0].view(torch.uint8), opt.v[0].view(torch.uint8), int(t)))
    assert all(torch.equal(a, b) for a, b in zip(results[0][:4], results[1][:4])) and results[0][4] == results[1][4] == 4


@pytest.mark.parametrize("bits", [32, 8])
def test_a_stacks_step_follows_its_gradients(bits):
    D, S, H, heads, F = 2, 256, 256, 4, 320
    weights = []
    for i in range(2):
        b = tsp_inputs.layer_inputs(tsp_inputs.LayerConfig("t", D, S, H, heads, F, 21 + i))
        w = {k: gu.dev(b[k]) for k in ("Wq", "Wk", "Wv", "Wo", "W1", "W3", "W2")}
        w["attn_norm"], w["mlp_norm"] = ((1 + 0.2 * normal(H, seed=i)).bfloat16() for _ in range(2))
        weights.append(w)
    stack = tsp.TSPStack(D, S, H, heads, F, weights, (1 + 0.2 * normal(H, seed=7)).bfloat16())
    stack.enable_updates(betas=BETAS, weight_decay=DECAY, state_bits=bits)
    xs, dout = normal(*stack.shape, seed=8).bfloat16(), normal(*stack.shape, seed=9).bfloat16()
    out, saved = stack.forward_train(xs)
    _, grads = stack.backward(saved, dout)
    kept = [g.clone() for g in grads]
    params = stack.wpack + stack.norms
    masters = [m for ms in stack.masters for m in ms]
    before = [m.double() for m in masters]
    assert all(torch.equal(p.float(), m) for p, m in zip(params, masters))
    total = stack.step(grads, LR, max_norm=0.5)
    assert all(torch.equal(a, b) for a, b in zip(kept, grads))
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    assert abs(float(total) - want) <= 1e-6 * want
    factor = min(1.0, 0.5 / (float(total) + 1e-6))
    for i, (p, m, w, g) in enumerate(zip(params, masters, before, grads)):
        g = g.double() * factor
        decay = DECAY if i < len(stack.wpack) else 0.0
        moved = LR * g / (g.abs() + 1e-8)  # the first step: m and v are corrected to g and g^2
        p1 = w - LR * decay * w - moved
        # in fp32: (1 - beta) g over its correction, off by 24 u; a g^2 below 2^-126 counts as zero in the root
        tol = U * p1.abs() + 24 * U * (moved.abs() + LR * decay * w.abs()) + 1e-12
        tol = torch.where(g.abs() < 1e-18, tol + LR * g.abs() / 1e-8, tol)
        assert bool(((m.double() - p1).abs() <= tol).all()), i
        assert torch.equal(p, m.bfloat16())
    again = stack.forward(xs)
    assert bool(torch.isfinite(again.float()).all()) and not torch.equal(again, out)
    stack.check()
