"""TSPAdamW against the update rule in 64 bits.

Tolerances, in units of u = 2^-24 (half a step of fp32): m and v are two products and a sum, three
roundings of terms no larger than the parts: 4 u of |b1 m| + |(1 - b1) g|. The update's quotient
takes m (4 u of its parts), the square root of v (its half, 2 u, and 2 u of its own), two products, a
sum and an approximate division (4 u): 16 u; the weight is rounded once more. The fp32 constants (betas, eps, rates) are
off by u each, which the 16 and the 4 include."""
import math

import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24
BETAS, EPS, DECAY, LR = (0.9, 0.95), 1e-8, 0.1, 3e-3


def blocks(n):
    return -(-n // 128)


def mix(x):
    x = ((x ^ (x >> 16)) * 0x7A35E9B5) & 0xFFFFFFFF
    x = ((x ^ (x >> 15)) * 0x68E31DA5) & 0xFFFFFFFF
    return x ^ (x >> 16)


def random_bits(n, seed, t, tensor, stream):
    key = mix((mix((mix((seed + t) & 0xFFFFFFFF) + tensor) & 0xFFFFFFFF) + stream) & 0xFFFFFFFF)
    return mix(torch.arange(n) ^ key)


def wide(codes, scales):
    n = codes.numel()
    return codes.float().double() * scales.double().repeat_interleave(128)[:n]


def rule(p, g, m, v, t, factor=1.0, lr=LR, decay=DECAY):
    """(p, m, v) after step t, and the terms that the tolerances go by."""
    b1, b2 = BETAS
    g = g * factor
    m1, v1 = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
    denominator = (v1 / (1 - b2 ** t)).sqrt() + EPS
    rate = lr / (1 - b1 ** t)
    parts = (b1 * m).abs() + ((1 - b1) * g).abs()
    return p - lr * decay * p - rate * m1 / denominator, m1, v1, parts, rate * parts / denominator + lr * decay * p.abs()


def within(got, want, tol):
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).max())


def pinned(low, high):
    """The check above left nearly every value one choice: about error / step of them, far below a
    hundredth, and the odd value next to zero have two."""
    assert int((low != high).sum()) <= 2 + low.numel() // 100


def check_states8(codes, scales, exact, parts, r16, keep):
    """The scale is the block's largest over 448; each code is the neighbour that the random bits
    choose, or the other one where the quotient lies within its own error of the border."""
    n = exact.numel()
    pad = torch.nn.functional.pad(exact, (0, -n % 128)).view(-1, 128)
    tops, tol = pad.abs().amax(1), torch.nn.functional.pad(parts, (0, -n % 128)).view(-1, 128).amax(1)
    want = torch.where(tops > 0, (tops / 448).clamp_min(2.0 ** -126), torch.ones_like(tops))
    within(scales, want, 5 * U * tol.clamp_min(0) / 448 + 2.0 ** -149)
    q = exact / scales.double().repeat_interleave(128)[:n]
    a = q.abs()
    step = torch.where(a < 2.0 ** -6, torch.full_like(a, 2.0 ** -9), 2.0 ** (torch.floor(torch.log2(a.clamp_min(1e-30))) - 3))
    error = 8 * U * parts / scales.double().repeat_interleave(128)[:n] + 2.0 ** -16 * step  # bits beyond the 16
    choose = lambda x: (torch.floor(x / step + r16.double() / 65536) * step).clamp(0, 448)  # noqa: E731
    low, high = choose((a - error).clamp_min(0)), choose(a + error)
    got = codes.float().double()
    mag = got.abs()
    if keep:
        low, high = [torch.where(exact > 0, x.clamp_min(2.0 ** -9), x) for x in (low, high)]
    assert bool(((mag >= low - 1e-12) & (mag <= high + 1e-12)).all())
    assert bool(((got == 0) | (got.sign() == exact.sign())).all())
    pinned(low, high)


def make(kinds, sizes, bits, seed, offset=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda k: torch.randn(k, generator=g)  # noqa: E731

    def place(x):  # offset: elements off the allocation's 16-byte boundary
        buf = torch.zeros(x.numel() + offset, dtype=x.dtype, device="cuda")[offset:]
        buf.copy_(x)
        return buf

    params, masters, grads = [], [], []
    for k, size in zip(kinds, sizes):
        w, grad = 0.1 * n(size), 0.01 * n(size)
        masters.append(place(w) if k == "master" else None)
        params.append(place(w if k == "fp32" else w.bfloat16()))
        grads.append(place(grad.bfloat16() if k == "bf16" else grad))
    opt = tsp.TSPAdamW(params, masters=masters, betas=BETAS, eps=EPS, weight_decay=DECAY, state_bits=bits, seed=5)
    m, v = [place(0.01 * n(s)) for s in sizes], [place((0.01 * n(s)).square()) for s in sizes]
    if bits == 8:
        out = []
        for xs in (m, v):
            codes, scales = [], []
            for x in xs:
                c = torch.zeros(1, x.numel(), dtype=E4M3, device="cuda")
                s = torch.zeros(1, blocks(x.numel()), device="cuda")
                tsp.tsp_quantize_e4m3(x[None], c, s)
                codes.append(place(c[0].view(torch.uint8)).view(E4M3))
                scales.append(s[0])
            out.append((codes, scales))
        opt.resume(40, out[0][0], out[1][0], out[0][1], out[1][1])
    else:
        opt.resume(40, m, v)
    return opt, params, masters, grads


def snapshot(opt, params, masters):
    """Weights (masters where there are any) and states as 64-bit values on the CPU."""
    w = [(b if b is not None else a).cpu().double() for a, b in zip(params, masters)]
    if opt.state_bits == 8:
        m = [wide(a.cpu(), s.cpu()) for a, s in zip(opt.m, opt.m_scales)]
        v = [wide(a.cpu(), s.cpu()) for a, s in zip(opt.v, opt.v_scales)]
    else:
        m, v = [x.cpu().double() for x in opt.m], [x.cpu().double() for x in opt.v]
    return w, m, v


def check_step(opt, params, masters, grads, kinds, before, t, factor=1.0, skipped=()):
    for i, kind in enumerate(kinds):
        if i in skipped:
            continue
        w, m, v = (x[i] for x in before)
        p1, m1, v1, parts, moved = rule(w, grads[i].cpu().double(), m, v, t, factor)
        if kind == "bf16":
            got = params[i].cpu().double()
            r = (random_bits(w.numel(), opt.seed, t, i, 1) & 0xFFFF).double() / 65536
            step = 2.0 ** (torch.floor(torch.log2(p1.abs().clamp_min(1e-30))) - 7)
            error = U * p1.abs() + 20 * U * moved
            low = torch.floor((p1.abs() - error) / step + r) * step
            high = torch.floor((p1.abs() + error) / step + r) * step
            assert bool(((got.abs() >= low) & (got.abs() <= high)).all())
            pinned(low, high)
        else:
            got = (params if kind == "fp32" else masters)[i]
            within(got.cpu(), p1, U * p1.abs() + 20 * U * moved + 1e-40)
            if kind == "master":
                assert torch.equal(params[i], masters[i].bfloat16())
        if opt.state_bits == 32:
            within(opt.m[i].cpu(), m1, 4 * U * parts + 1e-40)
            within(opt.v[i].cpu(), v1, 6 * U * v1 + 1e-40)
        else:
            r = random_bits(w.numel(), opt.seed, t, i, 0)
            check_states8(opt.m[i].cpu(), opt.m_scales[i].cpu(), m1, parts, r & 0xFFFF, False)
            check_states8(opt.v[i].cpu(), opt.v_scales[i].cpu(), v1, v1, r >> 16, True)


SIZES = [1, 7, 128, 129, 5000, 4096, 12289]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [0, 1, 3])
@pytest.mark.parametrize("kind", ["fp32", "bf16", "master"])
def test_a_step(kind, bits, offset):
    kinds = [kind] * len(SIZES)
    opt, params, masters, grads = make(kinds, SIZES, bits, 3, offset)
    for t in (41, 42):
        before = snapshot(opt, params, masters)
        opt.step(grads, LR)
        check_step(opt, params, masters, grads, kinds, before, t)
    assert opt.t == 42


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [1, 64, 65, 450])
def test_lists_of_many_lengths_and_kinds(count, bits):
    """Both tables, several launches of the large one, and tensors without a gradient."""
    kinds = [("fp32", "bf16", "master")[i % 3] for i in range(count)]
    sizes = [1 + (37 * i) % 400 for i in range(count)]
    opt, params, masters, grads = make(kinds, sizes, bits, count)
    before = snapshot(opt, params, masters)
    skipped = {i for i in range(count) if i % 100 == 50}
    saved = [params[i].clone() for i in skipped] + [opt.m[i].clone().view(torch.uint8) for i in skipped]
    opt.step([None if i in skipped else g for i, g in enumerate(grads)], LR)
    check_step(opt, params, masters, grads, kinds, before, 41, skipped=skipped)
    after = [params[i] for i in skipped] + [opt.m[i].view(torch.uint8) for i in skipped]
    assert all(torch.equal(a, b) for a, b in zip(saved, after))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("max_norm", [0.25, 1e9, math.inf, 0.0])
def test_clipping_on_the_way(max_norm, bits):
    kinds = ["fp32", "master"]
    opt, params, masters, grads = make(kinds, [4000, 333], bits, 8)
    norm = tsp.TSPGradClip(2).norm(grads)
    before = snapshot(opt, params, masters)
    opt.step(grads, LR, norm=norm, max_norm=max_norm)
    factor = min(1.0, max_norm / (float(norm) + 1e-6)) if math.isfinite(max_norm) else 1.0
    check_step(opt, params, masters, grads, kinds, before, 41, factor)


def test_from_zero_states():
    """The first step of a fresh optimizer moves every weight by lr: m and v are corrected alike."""
    for bits in (32, 8):
        p = torch.zeros(300, device="cuda")
        opt = tsp.TSPAdamW([p], betas=BETAS, state_bits=bits)
        g = torch.randn(300, generator=torch.Generator().manual_seed(2)).cuda() + 0.5
        opt.step([g], LR)
        assert torch.allclose(p, -LR * g.sign(), rtol=1e-5)


@pytest.mark.parametrize("eps", [1e-8, 1.2e-38])
def test_zero_gradients_and_states_leave_the_weights(eps):
    p = torch.randn(1000, device="cuda")
    before = p.clone()
    opt = tsp.TSPAdamW([p], eps=eps, state_bits=8)
    opt.step([torch.zeros(1000, device="cuda")], LR)
    assert torch.equal(p, before) and bool((opt.m_scales[0] == 1).all()) and bool((opt.v_scales[0] == 1).all())


def test_small_second_moments_are_never_lost():
    """An element far below its block's largest keeps a positive v: no step of m / eps."""
    p = torch.zeros(128, device="cuda")
    g = torch.full((128,), 1e-6, device="cuda")
    g[0] = 1.0
    opt = tsp.TSPAdamW([p], betas=BETAS, eps=1e-12, state_bits=8)
    for _ in range(20):
        opt.step([g], LR)
    assert bool((opt.v[0].float() > 0).all())
    assert float(p.abs().max()) <= 20 * LR * 1.01


def test_stochastic_rounding_follows_a_slow_mean():
    """v decays by 1 - beta2 a step without gradients; rounded to nearest it would stand still.
    Over 4096 blocks of equal values the mean keeps to the decay: each step's rounding has a
    variance of at most step^2 / 4, so the mean over 2^19 values after 60 steps is within 0.2 %."""
    n = 128 * 4096
    p = torch.zeros(n, device="cuda")
    opt = tsp.TSPAdamW([p], betas=(0.9, 0.999), state_bits=8, seed=3)
    v = torch.full((n,), 100.0, device="cuda").to(E4M3)
    v.view(4096, 128)[:, 0] = 448.0
    opt.resume(0, [torch.zeros(n, dtype=E4M3, device="cuda")], [v], [torch.ones(4096, device="cuda")],
               [torch.ones(4096, device="cuda")])
    start = v.float().view(4096, 128)[:, 1:].double().mean()
    for _ in range(60):
        opt.step([torch.zeros(n, device="cuda")], 0.0)
    now = (opt.v[0].float().view(4096, 128)[:, 1:] * opt.v_scales[0][:, None]).double().mean()
    assert abs(float(now / start) / 0.999 ** 60 - 1) < 0.002


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_counts_on(bits):
    """lr and t on the device: replays give the bits of eager steps."""
    kinds, sizes = ["fp32", "master", "bf16"], [500, 1000, 77]
    a = make(kinds, sizes, bits, 21)
    b = make(kinds, sizes, bits, 21)
    lr, t = torch.tensor(LR, device="cuda"), torch.tensor(41, device="cuda")
    norm = torch.tensor(3.0, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        b[0].step(b[3], lr, norm=norm, max_norm=1.0, t=t)
        t.add_(1)
    for k in range(3):
        a[0].step(a[3], torch.tensor(LR * (k + 1), device="cuda"), norm=norm, max_norm=1.0)
        lr.fill_(LR * (k + 1))
        graph.replay()
    torch.cuda.synchronize()
    assert int(t) == 44 and a[0].t == 43 and b[0].t == 40
    for x, y in zip(a[1] + a[0].m + a[0].v, b[1] + b[0].m + b[0].v):
        # device and host form 1 - beta^t with functions of their own: the same to a unit of fp32
        if x.dtype == torch.float32:
            assert torch.allclose(x, y, rtol=1e-6, atol=1e-12)
        else:
            assert (x.view(torch.uint8) != y.view(torch.uint8)).double().mean() < 0.01


def test_host_and_device_arguments_agree():
    kinds, sizes = ["fp32"], [5000]
    a, b = make(kinds, sizes, 32, 4), make(kinds, sizes, 32, 4)
    a[0].step(a[3], LR)
    b[0].step(b[3], torch.tensor(LR, device="cuda"), t=torch.tensor(41, device="cuda"))
    # the rates differ by a unit at most
    assert torch.allclose(a[1][0], b[1][0], rtol=0, atol=4 * U * 0.5)
    assert torch.equal(a[0].m[0], b[0].m[0])


def test_on_another_stream():
    kinds, sizes = ["fp32", "bf16"], [70000, 333]
    opt, params, masters, grads = make(kinds, sizes, 32, 6)
    before = snapshot(opt, params, masters)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    opt.step(grads, LR, stream=s)
    s.synchronize()
    check_step(opt, params, masters, grads, kinds, before, 41)
