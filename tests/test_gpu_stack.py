"""TSPStack (pre-norm layers, residual norm, clipping) and the operators around the layer in
one training step, against float64 torch with autograd.

Tolerance: relative Frobenius errors. A value rounded to bf16 is off by at most 2^-8 and by
2^-9 / sqrt(3) of its size in the root mean square for a uniform position in its binade, at
the worst 2^-9. A two-layer stack hands at most 16 rounded values one to the next in the
forward and 24 more in the backward; independent roundings add in squares, so the result is
within sqrt(40) 2^-9 = 1.3e-2 even if each passes on in full. TOL is 2e-2."""
import numpy as np
import pytest
import torch

import gpu_util as gu
import tsp_inputs

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu

TOL = 2e-2
EPS = 1e-5
NAMES = ("Wq", "Wk", "Wv", "Wo", "W1", "W3", "W2")


def rel(got, want):
    return float((got.double() - want).norm() / want.norm())


def norm64(h, w):
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * w


def layer64(h, w, heads):
    """One pre-norm layer on [sequences, S, H]."""
    B, S, H = h.shape
    y = norm64(h, w["attn_norm"])
    q, k, v = (torch.einsum("bsh,oh->bso", y, w[n]).view(B, S, heads, -1).transpose(1, 2)
               for n in ("Wq", "Wk", "Wv"))
    s = q @ k.transpose(-1, -2) / (H // heads) ** 0.5
    s = s.masked_fill(torch.ones(S, S, dtype=torch.bool, device=h.device).triu(1), -torch.inf)
    a = (torch.softmax(s, -1) @ v).transpose(1, 2).reshape(B, S, H)
    h = h + torch.einsum("bsh,oh->bso", a, w["Wo"])
    y = norm64(h, w["mlp_norm"])
    a1, a3 = (torch.einsum("bsh,oh->bso", y, w[n]) for n in ("W1", "W3"))
    return h + torch.einsum("bsf,of->bso", torch.nn.functional.silu(a1) * a3, w["W2"])


@pytest.mark.parametrize("stream_dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("shape", [(2, 256, 256, 4, 688, 1), (1, 200, 128, 2, 96, 1), (2, 256, 256, 2, 320, 2)], ids=str)
def test_stack_matches_autograd(shape, stream_dtype):
    D, S, H, heads, F, batch = shape
    layers = 2
    cfg = tsp_inputs.LayerConfig("t", D, S, H, heads, F, 21)
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    weights = []
    for i in range(layers):
        b = tsp_inputs.layer_inputs(tsp_inputs.LayerConfig("t", D, S, H, heads, F, 21 + i))
        w = {k: gu.dev(b[k]) for k in NAMES}
        # larger weights than the layer's workloads, so that each block matters beside its norm
        w = {k: (v.float() * 3).bfloat16() for k, v in w.items()}
        w["attn_norm"], w["mlp_norm"] = ((1 + 0.2 * n(H)).bfloat16() for _ in range(2))
        weights.append(w)
    last = (1 + 0.2 * n(H)).bfloat16()
    x, dout = n(batch, S, H).bfloat16(), n(batch, S, H).bfloat16()
    stack = tsp.TSPStack(D, S, H, heads, F, weights, last, eps=EPS, batch=batch, stream_dtype=stream_dtype)
    shard = lambda t: (tsp.tsp_shard(stack.plan, t, o := torch.empty_like(t)), o)[1]  # noqa: E731
    xs, gs = shard(x), shard(dout)
    out, saved = stack.forward_train(xs)
    plain = stack.forward(xs)
    assert torch.equal(plain, out) and torch.equal(xs, shard(x))
    dxs, grads = stack.backward(saved, gs)
    stack.check()

    w64 = [{k: v.double().requires_grad_() for k, v in w.items()} for w in weights]
    l64 = last.double().requires_grad_()
    x64 = x.double().requires_grad_()
    h = x64
    for w in w64:
        h = layer64(h, w, heads)
    want = norm64(h, l64)
    want.backward(dout.double())

    def unshard(t):
        o = torch.empty(t.shape, dtype=torch.bfloat16, device="cuda")
        tsp.tsp_unshard(stack.plan, t.bfloat16(), o)
        return o.view(batch, S, H)

    figures = {"out": rel(unshard(out), want.detach()), "dx": rel(unshard(dxs), x64.grad)}
    for i, w in enumerate(w64):
        parts = {"d" + k: torch.empty(v.shape, dtype=torch.float32, device="cuda") for k, v in w.items() if k in NAMES}
        tsp.tsp_unpack_weight_grads(stack.plan, grads[i], **parts)
        for k in NAMES:
            figures[f"layer {i} {k}"] = rel(parts["d" + k], w[k].grad)
        figures[f"layer {i} attn_norm"] = rel(grads[layers + 2 * i], w["attn_norm"].grad)
        figures[f"layer {i} mlp_norm"] = rel(grads[layers + 2 * i + 1], w["mlp_norm"].grad)
    figures["last_norm"] = rel(grads[-1], l64.grad)
    assert max(figures.values()) < TOL, figures

    # clipping: the norm over every true weight, in place
    before = [t.clone() for t in grads]
    total = sum(float((p.grad.double() ** 2).sum()) for w in w64 for p in w.values()) + float((l64.grad ** 2).sum())
    norm = stack.clip(grads, 0.5)
    assert abs(norm.item() - total ** 0.5) < TOL * total ** 0.5
    factor = min(1.0, 0.5 / (norm.item() + 1e-6))
    for a, b in zip(grads, before):
        assert torch.allclose(a, b * factor, rtol=1e-6, atol=0)


def test_stack_step_replays_from_a_graph():
    D, S, H, heads, F = 2, 256, 256, 4, 688
    b = tsp_inputs.layer_inputs(tsp_inputs.LayerConfig("t", D, S, H, heads, F, 3))
    w = {k: gu.dev(b[k]) for k in NAMES}
    w["attn_norm"] = w["mlp_norm"] = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    stack = tsp.TSPStack(D, S, H, heads, F, [w, w], w["attn_norm"])
    xs = gu.dev(b["x"])

    def step():
        out, saved = stack.forward_train(xs)
        dxs, grads = stack.backward(saved, out)
        return (out, dxs, stack.clip(grads, 1.0), *grads)

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(2):
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    stack.check()


def test_operators_together_on_a_packed_batch():
    """One attention block over a packed batch with grouped heads, as a user composes it: norm,
    projections, packed attention, output projection, residual norm; backward; clipping."""
    H, heads, kv, d = 256, 8, 2, 64
    lengths = [1, 130, 40, 0, 77]
    starts_host = [0] + list(np.cumsum(lengths))
    T = int(starts_host[-1])
    g = torch.Generator(device="cuda")
    g.manual_seed(8)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dy2, dh2 = n(T, H).bfloat16(), n(T, H).bfloat16(), n(T, H)
    stream = 2 * n(T, H)
    wqkv = (n((heads + 2 * kv) * d, H) / 16).bfloat16()
    wo = (n(H, heads * d) / 16).bfloat16()
    w1, w2 = ((1 + 0.2 * n(H)).bfloat16() for _ in range(2))
    starts = torch.tensor(starts_host, dtype=torch.int32, device="cuda")
    norm = tsp.TSPRMSNorm(T, H, eps=EPS)
    att = tsp.TSPPackedAttention(T, len(lengths), heads, kv, d)
    clip = tsp.TSPGradClip(4)

    y1, h1 = norm.forward(x, w1, residual=stream)
    qkv = y1 @ wqkv.T
    split = lambda t: (t[:, :heads * d].unflatten(1, (heads, d)),  # noqa: E731
                       t[:, heads * d:(heads + kv) * d].unflatten(1, (kv, d)),
                       t[:, (heads + kv) * d:].unflatten(1, (kv, d)))
    q, k, v = split(qkv)
    o, lse = att.forward_train(q, k, v, starts)
    a = o.view(T, -1) @ wo.T
    y2, h2 = norm.forward(a, w2, residual=h1)
    # backward
    da = torch.empty_like(a)
    dh1, dw2 = norm.backward(h2, w2, dy2, dh=dh2, dx16=da)
    do = (da @ wo).view(T, heads, d)
    dwo = (da.T.float() @ o.view(T, -1).float())
    dqkv = torch.empty_like(qkv)
    att.backward(q, k, v, starts, o, lse, do, *split(dqkv))
    dy1 = dqkv @ wqkv
    dwqkv = dqkv.T.float() @ y1.float()
    dx, dw1 = norm.backward(h1, w1, dy1, dh=dh1)
    att.check()

    X, Sm = x.double().requires_grad_(), stream.double()
    P = {k_: t.double().requires_grad_() for k_, t in (("wqkv", wqkv), ("wo", wo), ("w1", w1), ("w2", w2))}
    H1 = X + Sm
    QKV = norm64(H1, P["w1"]) @ P["wqkv"].T
    Q, K, V = split(QKV)
    outs = []
    for s0, s1 in zip(starts_host, starts_host[1:]):
        L = int(s1 - s0)
        f = lambda t, r: t[s0:s1].transpose(0, 1).repeat_interleave(r, 0)  # noqa: E731
        sc = f(Q, 1) @ f(K, heads // kv).transpose(1, 2) / d ** 0.5
        sc = sc.masked_fill(torch.ones(L, L, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
        outs.append((torch.softmax(sc, -1) @ f(V, heads // kv)).transpose(0, 1))
    H2 = H1 + torch.cat(outs).reshape(T, -1) @ P["wo"].T
    Y2 = norm64(H2, P["w2"])
    ((Y2 * dy2.double()).sum() + (H2 * dh2.double()).sum()).backward()
    figures = {"y2": rel(y2, Y2.detach()), "h2": rel(h2, H2.detach()), "dx": rel(dx, X.grad)}
    for name, got in (("wqkv", dwqkv), ("wo", dwo), ("w1", dw1), ("w2", dw2)):
        figures[name] = rel(got, P[name].grad)
    assert max(figures.values()) < TOL, figures
    grads = [dwqkv, dwo, dw1, dw2]
    total = sum(float((t.grad ** 2).sum()) for t in P.values()) ** 0.5
    before = [t.clone() for t in grads]
    got = clip.clip(grads, 0.25 * total).item()
    assert abs(got - total) < TOL * total
    for t, b in zip(grads, before):
        assert torch.allclose(t, b * (0.25 * total / (got + 1e-6)), rtol=1e-6, atol=0)
