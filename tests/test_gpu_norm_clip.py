"""Residual RMS norm (bf16 and e4m3 outputs, backward) and gradient clipping on the GPU,
against the formulas in float64.

Tolerances. A rounding to a type is off by at most half a step: 2^-8 relative for bf16,
2^-24 for fp32, and for e4m3 half of 2^(max(e, -6) - 3) at a value in [2^e, 2^(e+1)).
The fp32 sums of a row take at most 32 elements one after the other in a thread and ten
levels of a tree, each step off by 2^-24 of the sum of magnitudes; with the square root,
the reciprocal and the products that is below SUM = 64 * 2^-24 relative for sums of
positive terms."""
import math

import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu

SUM = 64 * 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
EPS = 1e-5

WIDTHS = [1, 7, 8, 128, 130, 256, 1000, 1001, 1024, 1032, 4096, 4095, 16384, 16392, 20001, 32768]


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def within(got, want, bound, what):
    got, want = got.double(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.isfinite(got).all(), what
    worst = ((got - want).abs() - bound).max().item() if got.numel() else -1.0
    assert worst <= 0, f"{what}: {worst:.3e} over the bound"


def exact_norm(x, r, w, eps=EPS):
    h = x.double() + (0 if r is None else r.double())
    y = h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w.double()
    return h, y


def check_e4m3(y8, scales, y, group, what):
    rows, width = y.shape
    g = group or width
    groups = -(-width // g)
    top = torch.nn.functional.pad(y.abs(), (0, groups * g - width)).view(rows, groups, g).amax(-1)
    want = torch.where(top > 0, (top / 448).clamp_min(2.0 ** -126), torch.ones_like(top))
    within(scales, want, 2 * SUM * want, what + " scales")
    t = y / scales.double().repeat_interleave(g, 1)[:, :width]
    step = torch.exp2(torch.log2(t.abs().clamp_min(2.0 ** -6)).floor() - 3)
    within(y8.float(), t, step / 2 + 2 * SUM * t.abs(), what + " y8")


@pytest.mark.parametrize("rows", [1, 3, 700])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_forward(rows, width):
    n = gen(rows * 100003 + width)
    x = (n(rows, width) * torch.exp(n(width))).bfloat16()
    w = (1 + 0.3 * n(width)).bfloat16()
    op = tsp.TSPRMSNorm(rows, width, eps=EPS)
    for kind in (None, torch.bfloat16, torch.float32):
        r = None if kind is None else (2 * n(rows, width)).to(kind)
        eh, ey = exact_norm(x, r, w)
        y, h = op.forward(x, w, residual=r)
        tag = f"{rows}x{width} {kind}"
        within(y, ey, (HALF[torch.bfloat16] + SUM) * ey.abs() + 2.0 ** -133, tag + " y")
        if kind is None:
            assert h is None
        else:
            # one fp32 addition, then the rounding to h's type
            within(h, eh, (HALF[kind] + 2.0 ** -23) * eh.abs() + 2.0 ** -133, tag + " h")
        for group in (0, 128):
            y8, sc, h8 = op.forward_e4m3(x, w, residual=r, group=group)
            check_e4m3(y8, sc, ey, group, f"{tag} group {group}")
            if h is not None:
                assert torch.equal(h, h8)


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
def test_norm_forward_in_place_and_unaligned(kind):
    """h over the residual, y over x; buffers that start off a 16-byte boundary."""
    n = gen(5)
    rows, width = 37, 1024
    w = (1 + 0.3 * n(width + 1)).bfloat16()[1:]
    x = n(rows * width + 1).bfloat16()[1:].view(rows, width)
    r = n(rows * width + 1).to(kind)[1:].view(rows, width)
    op = tsp.TSPRMSNorm(rows, width)
    y0, h0 = op.forward(x.clone(), w.clone(), residual=r.clone())
    y, h = op.forward(x, w, residual=r, y=x, h=r)
    assert y.data_ptr() == x.data_ptr() and h.data_ptr() == r.data_ptr()
    # the 16-byte and the single-element path sum in another order
    within(y, y0, 2.0 ** -7 * y0.double().abs(), "unaligned y")
    assert torch.equal(h, h0)
    xa, ra = x.clone(), r.clone()
    y1, h1 = op.forward(xa.clone(), w.clone(), residual=ra.clone())
    y2, h2 = op.forward(xa, w.clone(), residual=ra, y=xa, h=ra)
    assert torch.equal(y1, y2) and torch.equal(h1, h2)


def test_norm_special_rows():
    """Zero rows, tiny and huge values, infinities and NaN stay in their own rows."""
    n = gen(9)
    width = 1000
    x = n(8, width).bfloat16()
    x[1] = 0
    x[2] = 1e-30
    x[3] = 1e15
    x[4, 17] = math.inf
    x[5, 3] = math.nan
    w = (1 + 0.3 * n(width)).bfloat16()
    op = tsp.TSPRMSNorm(8, width, eps=EPS)
    y, _ = op.forward(x, w)
    _, ey = exact_norm(x, None, w)
    for i in (0, 1, 2, 3, 6, 7):
        within(y[i], ey[i], (HALF[torch.bfloat16] + SUM) * ey[i].abs() + 2.0 ** -133, f"row {i}")
    assert torch.isnan(y[5]).all() and torch.isnan(y[4, 17])
    for group in (0, 128):
        y8, sc, _ = op.forward_e4m3(x, w, group=group)
        good = [0, 1, 2, 3, 6, 7]
        check_e4m3(y8[good], sc[good], ey[good], group, f"special rows, group {group}")
        assert (sc[1] == 1).all() and (y8[1].float() == 0).all()
        assert torch.isnan(sc[5, 0])


def exact_norm_bwd(h, w, dy, dh, eps=EPS):
    """(dx, bound on its sums' error, dw, its sum of magnitudes) in float64."""
    h, w, dy = h.double(), w.double(), dy.double()
    n = h.shape[1]
    rstd = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    g = dy * w
    dx = rstd * g - h * rstd ** 3 * (g * h).sum(-1, keepdim=True) / n
    mag = rstd * g.abs() + h.abs() * rstd ** 3 * (g * h).abs().sum(-1, keepdim=True) / n
    if dh is not None:
        dx, mag = dx + dh.double(), mag + dh.double().abs()
    t = dy * h * rstd
    return dx, mag, t.sum(0), t.abs().sum(0)


@pytest.mark.parametrize("rows", [1, 5, 1300])
@pytest.mark.parametrize("width", WIDTHS)
def test_norm_backward(rows, width):
    n = gen(rows * 7 + width)
    w = (1 + 0.3 * n(width)).bfloat16()
    dy = n(rows, width).bfloat16()
    op = tsp.TSPRMSNorm(rows, width, eps=EPS)
    # rows of a CTA (of 152 at least) and of its eight warps one after the other, then up to 456
    # partial rows in 32 chains and a tree
    dw_steps = 64 + math.ceil(rows / 152) + 8 + 456 / 32 + 5
    for kind in (torch.bfloat16, torch.float32):
        h = (3 * n(rows, width) * torch.exp(n(width))).to(kind)
        for dh in (None, n(rows, width).to(kind)):
            dx, dw = op.backward(h, w, dy, dh=dh)
            edx, mag, edw, dmag = exact_norm_bwd(h, w, dy, dh)
            tag = f"{rows}x{width} {kind} dh={dh is not None}"
            within(dx, edx, HALF[kind] * edx.abs() + SUM * mag + 2.0 ** -133, tag + " dx")
            within(dw, edw, dw_steps * 2.0 ** -24 * dmag + 2.0 ** -133, tag + " dw")
            dx16 = torch.empty_like(dy)
            dx2, dw2 = op.backward(h, w, dy, dh=dh, dx16=dx16)
            assert torch.equal(dx, dx2) and torch.equal(dw, dw2)  # the same bits every time
            assert torch.equal(dx16, dx.bfloat16())


def test_norm_backward_matches_differences():
    """dx and dw against central differences of the definition in float64."""
    n = gen(31)
    rows, width = 2, 24
    h = n(rows, width)
    w, dy = (1 + 0.3 * n(width)).bfloat16(), n(rows, width).bfloat16()
    op = tsp.TSPRMSNorm(rows, width, eps=EPS)
    dx, dw = op.backward(h, w, dy)

    def loss(hh, ww):
        hh, ww = hh.double(), ww.double()
        return (hh / torch.sqrt((hh * hh).mean(-1, keepdim=True) + EPS) * ww * dy.double()).sum()

    step = 1e-4  # the differences' own error is of order step^2
    for i in range(rows):
        for j in range(width):
            d = torch.zeros(rows, width, dtype=torch.float64, device="cuda")
            d[i, j] = step
            want = (loss(h.double() + d, w) - loss(h.double() - d, w)) / (2 * step)
            assert abs(dx[i, j].item() - want.item()) < 1e-5
    for j in range(width):
        d = torch.zeros(width, dtype=torch.float64, device="cuda")
        d[j] = step
        want = (loss(h, w.double() + d) - loss(h, w.double() - d)) / (2 * step)
        assert abs(dw[j].item() - want.item()) < 1e-5


@pytest.mark.parametrize("width", [1024, 4096, 8192])
def test_norm_backward_with_and_without_dh_in_turn(width):
    """The two take different amounts of shared memory in one kernel."""
    n = gen(width)
    rows = 40
    h, dh = n(rows, width).bfloat16(), n(rows, width).bfloat16()
    w, dy = (1 + 0.3 * n(width)).bfloat16(), n(rows, width).bfloat16()
    op = tsp.TSPRMSNorm(rows, width, eps=EPS)
    first = [op.backward(h, w, dy, dh=d) for d in (dh, None)]
    for _ in range(2):
        for d, (dx, dw) in zip((dh, None), first):
            dx2, dw2 = op.backward(h, w, dy, dh=d)
            assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_norm_no_rows():
    op = tsp.TSPRMSNorm(4, 64)
    x = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    y, h = op.forward(x, w)
    assert y.shape == (0, 64) and h is None
    dx, dw = op.backward(x, w, x)
    assert dx.shape == (0, 64) and (dw == 0).all()


# ------------------------------------------------------------------ gradient clipping

def exact_clip(grads, max_norm):
    total = sum(float((g.double() ** 2).sum()) for g in grads)
    norm = math.sqrt(total)
    return norm, [g.double() * min(1.0, max_norm / (norm + 1e-6)) for g in grads]


def check_clip(grads, max_norm, outs, norm, what):
    enorm, eouts = exact_clip(grads, max_norm)
    # 16 squares one after the other and two levels in fp32, the rest in fp64, one rounding
    rel = 20 * 2.0 ** -24
    assert abs(norm.item() - enorm) <= rel * enorm, (what, norm.item(), enorm)
    for i, (g, o, e) in enumerate(zip(grads, outs, eouts)):
        within(o, e, (HALF[g.dtype] + 2 * rel) * e.abs() + 2.0 ** -133, f"{what} tensor {i}")


SIZES = {
    "one": [1],
    "tails": [1, 2, 3, 5, 8, 255, 256, 257, 16383, 16384, 16385, 100001],
    "empty": [0, 7, 0, 40000, 0],
    "many": [(i * 37) % 900 + 1 for i in range(200)],
    "over a thousand": [(i * 13) % 50 + 1 for i in range(2500)],
    "large": [3_000_001, 5_000_000],
}


@pytest.mark.parametrize("sizes", list(SIZES), ids=list(SIZES))
@pytest.mark.parametrize("max_norm", [0.5, 1e9, math.inf, 0.0])
def test_clip(sizes, max_norm):
    n = gen(len(sizes))
    grads = [(n(s) * 10.0 ** -(i % 4)).to(torch.bfloat16 if i % 3 == 1 else torch.float32)
             for i, s in enumerate(SIZES[sizes])]
    op = tsp.TSPGradClip(len(grads))
    outs = [torch.full_like(g, 7) for g in grads]
    before = [g.clone() for g in grads]
    norm = op.clip(grads, max_norm, outs=outs)
    check_clip(grads, max_norm, outs, norm, sizes)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    assert torch.equal(op.norm(grads), norm)
    again = op.clip(grads, max_norm)  # in place: the same bits
    assert torch.equal(again, norm) and all(torch.equal(a, b) for a, b in zip(grads, outs))


def test_clip_unaligned_views():
    n = gen(3)
    flat32, flat16 = n(50000), n(50000).bfloat16()
    grads = [flat32[1:20002], flat32[30001:30002], flat16[3:40003], flat16[40005:40006]]
    outs = [torch.empty(g.numel() + 1, dtype=g.dtype, device="cuda")[1:] for g in grads]
    op = tsp.TSPGradClip(4)
    norm = op.clip(grads, 0.25, outs=outs)
    check_clip(grads, 0.25, outs, norm, "unaligned")


@pytest.mark.parametrize("size", [1e25, 3e38, 1e-25, 1e-40])
def test_clip_whole_range(size):
    """Squares that overflow or vanish in fp32."""
    n = gen(11)
    g = (n(40000).clamp(-1, 1) * size).float()
    norm = tsp.TSPGradClip(1).norm([g])
    want = math.sqrt(float((g.double() ** 2).sum()))
    if want > torch.finfo(torch.float32).max:
        assert math.isinf(norm.item())
        out = torch.empty_like(g)
        tsp.TSPGradClip(1).clip([g], 1.0, outs=[out])
        within(out, g.double() / want, 2.0 ** -22 * g.double().abs() / want + 2.0 ** -149, "huge")
    else:
        assert abs(norm.item() - want) <= 20 * 2.0 ** -24 * want + 2.0 ** -149


def test_clip_non_finite():
    op = tsp.TSPGradClip(2)
    a, b = torch.ones(100, device="cuda"), torch.ones(30000, device="cuda")
    b[77] = math.inf
    outs = [torch.empty_like(a), torch.empty_like(b)]
    assert math.isinf(op.clip([a, b], 1.0, outs=outs).item())
    assert (outs[0] == 0).all() and torch.isnan(outs[1][77]) and (outs[1][:77] == 0).all()
    b[78] = math.nan
    assert math.isnan(op.clip([a, b], 1.0, outs=outs).item())
    assert torch.isnan(outs[0]).all() and torch.isnan(outs[1]).all()


def test_clip_refuses_overlaps():
    x = torch.ones(1000, device="cuda")
    y = torch.ones(1000, device="cuda")
    op = tsp.TSPGradClip(3)
    for grads, outs in [([x, x], [x, x]), ([x, y], [y, x]), ([x, y], [y, torch.empty_like(y)]),
                        ([x[:500], x[499:999]], None), ([x[:500]], [x[1:501]])]:
        with pytest.raises(tsp.TSPError) as e:
            op.clip(grads, 1.0, outs=outs)
        assert e.value.status == tsp.TSP_ERR_INVALID_ARG and "overlaps" in str(e.value)
    assert (x == 1).all() and (y == 1).all()
    # the same gradient twice, to two outputs, counts twice
    outs = [torch.empty_like(x), torch.empty_like(x)]
    norm = op.clip([x, x], 1.0, outs=outs)
    check_clip([x, x], 1.0, outs, norm, "twice")


# ------------------------------------------------------------------ streams and graphs

def test_norm_and_clip_replay_from_a_graph_on_another_stream():
    n = gen(77)
    rows, width = 300, 1024
    x, r = n(rows, width).bfloat16(), n(rows, width)
    w, dy = (1 + 0.1 * n(width)).bfloat16(), n(rows, width).bfloat16()
    norm_op, clip_op = tsp.TSPRMSNorm(rows, width), tsp.TSPGradClip(2)

    def step():
        y, h = norm_op.forward(x, w, residual=r)
        dx, dw = norm_op.backward(h, w, dy, dh=h)
        norm = clip_op.clip([dx, dw], 0.1)
        return y, h, dx, dw, norm

    eager = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    torch.cuda.current_stream().wait_stream(side)
    x2, r2 = n(rows, width).bfloat16(), n(rows, width)
    keep = x.clone(), r.clone()
    x.copy_(x2)
    r.copy_(r2)
    graph.replay()
    want = [t.clone() for t in step()]
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    x.copy_(keep[0])
    r.copy_(keep[1])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))
    torch.cuda.synchronize()
    # an explicit stream argument
    y, _ = norm_op.forward(x, w, residual=r, stream=side)
    side.synchronize()
    assert torch.equal(y, eager[0])


def test_no_clipping_of_an_infinite_norm():
    """max_norm infinite: the gradients stay as they are, whatever the norm but NaN."""
    op = tsp.TSPGradClip(2)
    a = torch.tensor([1.0, math.inf, -3.0], device="cuda")
    b = torch.tensor([2.0, -4.0], device="cuda", dtype=torch.bfloat16)
    outs = [torch.zeros_like(a), torch.zeros_like(b)]
    assert math.isinf(op.clip([a, b], math.inf, outs=outs).item())
    assert torch.equal(outs[0], a) and torch.equal(outs[1], b)
    a[1] = math.nan
    assert math.isnan(op.clip([a, b], math.inf, outs=outs).item())
    assert torch.isnan(outs[0]).all() and torch.isnan(outs[1]).all()
