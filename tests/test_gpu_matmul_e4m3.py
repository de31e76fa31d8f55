"""tsp_matmul_e4m3 and TSPLinearE4M3 against the same sums in 64 bits.

Tolerance of an output: a block's products of e4m3 values are exact and are summed in fp32 by the tensor
cores, 128 of them: at most 128 u relative to the sum of their magnitudes (u = 2^-24). The product of
two scales, the scaling and the sum over the blocks add (2 + 1 + number of blocks) u; the orders
that split the blocks do not exceed that. A bf16 result is rounded once more, half a step 2^-8 of its value."""
import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24


def blocks(n):
    return -(-n // 128)


def operand(rows, k, seed, block, ld=None, decades=2):
    """(e4m3 [rows, k] in rows of ld bytes, scales): every code but NaN, scales over some decades. What lies
    behind the rows is NaN."""
    g = torch.Generator().manual_seed(seed)
    ld = -(-k // 16) * 16 if ld is None else ld
    buf = torch.full((rows, ld), 0x7F, dtype=torch.uint8)
    # small values mostly, as quantised normal numbers have them, and some of any size
    x = (torch.randn(rows, k, generator=g) * 60).clamp(-448, 448).to(E4M3).view(torch.uint8)
    any_code = torch.randint(0, 256, (rows, k), generator=g).to(torch.uint8)
    any_code[(any_code & 0x7F) == 0x7F] = 0
    buf[:, :k] = torch.where(torch.rand(rows, k, generator=g) < 0.05, any_code, x)
    scales = 10 ** (decades * (torch.rand(-(-rows // block), blocks(k), generator=g) - 0.5))
    return buf.cuda().view(E4M3)[:, :k], scales.cuda()


def wide(x, scales, block):
    s = scales.double().repeat_interleave(128, 1)[:, :x.shape[1]]
    if block == 128:
        s = s.repeat_interleave(128, 0)[:x.shape[0]]
    return x.float().double() * s


def expected(a, sa, b, sb, b_block):
    """The product, and the sum of the terms' magnitudes."""
    x, y = wide(a, sa, 1), wide(b, sb, b_block)
    return x @ y.t(), x.abs() @ y.abs().t()


def within(got, want, size, k, extra=0.0):
    tol = (128 + 3 + blocks(k)) * U * size + extra
    if got.dtype == torch.bfloat16:
        tol = tol + (want.abs() + tol) * 2.0 ** -8
    off = (got.double() - want).abs()
    assert bool((off <= tol).all()), float((off / tol.clamp_min(1e-300)).max())


@pytest.fixture(scope="module")
def ws():
    t = torch.zeros(tsp.tsp_matmul_e4m3_workspace_bytes(), dtype=torch.uint8, device="cuda")
    yield t
    assert tsp.tsp_device_status(t) == tsp.TSP_OK


def run(m, n, k, b_block, dtype, ws, seed=0, accumulate=False, pad_c=0, base_c=0):
    a, sa = operand(m, k, seed + 1, 1)
    b, sb = operand(n, k, seed + 2, b_block)
    flat = torch.full((m * (n + pad_c) + base_c,), 7.5, dtype=dtype, device="cuda")
    c = flat[base_c:].view(m, n + pad_c)
    tsp.tsp_matmul_e4m3(a, sa, b, sb, c[:, :n], ws, b_block=b_block, accumulate=accumulate)
    want, size = expected(a, sa, b, sb, b_block)
    extra = 0.0
    if accumulate:
        want, extra = want + 7.5, U * (want.abs() + 7.5)
    within(c[:, :n], want, size, k, extra)
    assert bool((c[:, n:] == 7.5).all()) and bool((flat[:base_c] == 7.5).all())


# one row to some tiles, every tile width, splits of K from 1 to 8, ends inside a tile or a block
SHAPES = [(1, 1, 1), (1, 128, 128), (1, 4096, 1024), (3, 129, 127), (16, 500, 2048), (17, 1000, 4096), (33, 64, 520),
          (64, 256, 1000), (100, 688, 256), (128, 128, 4096), (129, 257, 384), (200, 1001, 1001), (300, 64, 64),
          (1000, 1024, 300), (2000, 1300, 520), (1300, 2816, 128), (5000, 520, 130)]


@pytest.mark.parametrize("b_block", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("m, n, k", SHAPES)
def test_products(m, n, k, dtype, b_block, ws):
    run(m, n, k, b_block, dtype, ws, seed=m + n + k)


# K split over clusters of 3, 5, 6, 7 and 8; tiles that walk in groups of rows (b above 48 MB)
@pytest.mark.parametrize("m, n, k", [(4, 11000, 1024), (2, 7680, 1280), (30, 6400, 1536), (9, 5500, 1800), (50, 2400, 2048),
                                     (600, 13000, 4096)])
def test_splits_and_tile_orders(m, n, k, ws):
    run(m, n, k, 128, torch.bfloat16, ws, seed=n)


@pytest.mark.parametrize("dtype, n, pad", [(torch.bfloat16, 1, 7), (torch.bfloat16, 9, 7), (torch.float32, 3, 1),
                                           (torch.float32, 1, 3), (torch.bfloat16, 130, 6)])
def test_narrow_outputs_of_many_rows(dtype, n, pad, ws):
    """Rows that end inside 16 bytes: what lies behind them stays."""
    for b_block in (1, 128):
        run(30000, n, 256, b_block, dtype, ws, pad_c=pad)


@pytest.mark.parametrize("m, n, k", [(5, 300, 4096), (700, 4096, 256), (1, 1, 1)])
def test_adding_to_the_output(m, n, k, ws):
    run(m, n, k, 1, torch.float32, ws, accumulate=True)
    run(m, n, k, 128, torch.float32, ws, accumulate=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("pad, base", [(0, 1), (3, 0), (8, 8), (16, 16)])
@pytest.mark.parametrize("m, n", [(20, 200), (3000, 1024)])
def test_output_strides_and_offsets(m, n, pad, base, dtype, ws):
    run(m, n, 256, 128, dtype, ws, pad_c=pad, base_c=base)


def test_wide_row_strides_of_the_operands(ws):
    a, sa = operand(130, 200, 1, 1, ld=1024)
    b, sb = operand(70, 200, 2, 128, ld=208)
    c = torch.empty(130, 70, device="cuda")
    tsp.tsp_matmul_e4m3(a, sa, b, sb, c, ws)
    within(c, *expected(a, sa, b, sb, 128), 200)


def test_empty(ws):
    for m, n, k in ((0, 5, 128), (5, 0, 128), (5, 7, 0)):
        a, sa = operand(m, k, 1, 1)
        b, sb = operand(n, k, 2, 128)
        c = torch.full((m, n), 3.0, device="cuda")
        tsp.tsp_matmul_e4m3(a, sa, b, sb, c, ws)
        assert bool((c == 0).all())
        c.fill_(3.0)
        tsp.tsp_matmul_e4m3(a, sa, b, sb, c, ws, accumulate=True)
        assert bool((c == 3).all())


@pytest.mark.parametrize("m, n", [(4, 300), (2000, 1200)])
def test_a_bad_scale_stays_in_its_rows(m, n, ws):
    a, sa = operand(m, 512, 1, 1)
    b, sb = operand(n, 512, 2, 128)
    clean = torch.empty(m, n, device="cuda")
    tsp.tsp_matmul_e4m3(a, sa, b, sb, clean, ws)
    sa[2, 1], sb[1, 0] = float("nan"), float("inf")
    c = torch.empty(m, n, device="cuda")
    tsp.tsp_matmul_e4m3(a, sa, b, sb, c, ws)
    hit = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    hit[2] = True
    hit[:, 128:256] = True
    assert bool((~torch.isfinite(c[hit])).all()) and torch.equal(c[~hit], clean[~hit])


def test_the_same_bits_every_time(ws):
    for m, n, k in ((7, 600, 4096), (1500, 2000, 384)):
        a, sa = operand(m, k, 1, 1)
        b, sb = operand(n, k, 2, 1)
        c = [torch.empty(m, n, device="cuda") for _ in range(3)]
        for x in c:
            tsp.tsp_matmul_e4m3(a, sa, b, sb, x, ws, b_block=1)
        assert torch.equal(c[0], c[1]) and torch.equal(c[0], c[2])


# ------------------------------------------------------------------ TSPLinearE4M3

def quantised(x):
    """What x stands for after tsp_quantize_e4m3 by rows (tested bit for bit on its own)."""
    q = torch.empty(x.shape, dtype=E4M3, device="cuda")
    s = torch.empty(x.shape[0], blocks(x.shape[1]), device="cuda")
    tsp.tsp_quantize_e4m3(x, q, s)
    return wide(q, s, 1)


def normal(*shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).cuda()


@pytest.mark.parametrize("tokens, n, k", [(1, 1, 1), (5, 300, 100), (130, 256, 688), (1000, 520, 384)])
def test_a_training_step_of_a_layer(tokens, n, k):
    layer = tsp.TSPLinearE4M3(tokens + 3, n, k)
    w = layer.quantize_weight(0.05 * normal(n, k, seed=1))
    x, dy = normal(tokens, k, seed=2).bfloat16(), normal(tokens, n, seed=3).bfloat16()
    y, saved = layer.forward_train(x, w)
    assert torch.equal(y, layer.forward(x, w))
    dx, dw = layer.backward(saved, dy, w)
    w64, x64, dy64 = wide(w.values, w.scales, 128), quantised(x), quantised(dy)
    within(y, x64 @ w64.t(), x64.abs() @ w64.abs().t(), k)
    within(dx, dy64 @ w64, dy64.abs() @ w64.abs(), n)
    xt, dyt = quantised(x.t().contiguous()), quantised(dy.t().contiguous())
    want, size = dyt @ xt.t(), dyt.abs() @ xt.abs().t()
    within(dw, want, size, tokens)
    again = dw.clone()
    layer.backward(saved, dy, w, dw=again, accumulate=True)
    assert torch.equal(again, dw + dw)
    layer.check()


def test_the_norms_output_is_an_input():
    tokens, n, k = 40, 300, 512
    layer, norm = tsp.TSPLinearE4M3(tokens, n, k), tsp.TSPRMSNorm(tokens, k)
    w = layer.quantize_weight(0.05 * normal(n, k, seed=1).bfloat16(), training=False)
    assert w.values_t is None
    x8, scales, _ = norm.forward_e4m3(normal(tokens, k, seed=2).bfloat16(), torch.ones(k, dtype=torch.bfloat16, device="cuda"))
    y = layer.forward(x8, w, scales=scales)
    x64, w64 = wide(x8, scales, 1), wide(w.values, w.scales, 128)
    within(y, x64 @ w64.t(), x64.abs() @ w64.abs().t(), k)


def test_gradients_are_those_of_the_function():
    """Against differences of the layer's own forward, for a loss sum(y dy). Quantising moves x and w by up to
    2^-4 of a value: the inputs are powers of two, which e4m3 holds exactly, and so is the step."""
    tokens, n, k = 6, 140, 130
    g = torch.Generator().manual_seed(7)
    powers = lambda *s: (2.0 ** torch.randint(0, 4, s, generator=g) * (torch.randint(0, 2, s, generator=g) * 2 - 1)).cuda()  # noqa: E731
    layer = tsp.TSPLinearE4M3(tokens, n, k)
    x, w, dy = powers(tokens, k), powers(n, k), powers(tokens, n)
    x[:, 0], w[:, 0], x[:, 128], w[0] = 8, 8, 8, 8  # the largest of every block stays the same
    weight = layer.quantize_weight(w)
    y, saved = layer.forward_train(x.bfloat16(), weight)
    dx, dw = layer.backward(saved, dy.bfloat16(), weight)
    loss = lambda x, w: (x.double() @ w.double().t() * dy.double()).sum()  # noqa: E731
    for _ in range(20):
        i, j = int(torch.randint(0, tokens, (1,), generator=g)), int(torch.randint(1, 128, (1,), generator=g))
        up = x.clone()
        up[i, j] += 1
        want = float(loss(up, w) - loss(x, w))
        assert abs(float(dx[i, j]) - want) <= abs(want) * 2.0 ** -8
        r = int(torch.randint(1, n, (1,), generator=g))
        up = w.clone()
        up[r, j] += 1
        assert abs(float(dw[r, j]) - float(loss(x, up) - loss(x, w))) <= 1e-3


def test_a_captured_step_is_replayed_and_keeps_its_workspace():
    tokens, n, k = 70, 200, 300
    layer = tsp.TSPLinearE4M3(tokens, n, k)
    w = layer.quantize_weight(0.05 * normal(n, k, seed=1))
    x, dy = normal(tokens, k, seed=2).bfloat16(), normal(tokens, n, seed=3).bfloat16()
    forward = torch.cuda.CUDAGraph()
    layer.forward(x, w)
    torch.cuda.synchronize()
    with torch.cuda.graph(forward):
        y1 = layer.forward(x, w)
    layer.enable_backward()
    step = torch.cuda.CUDAGraph()
    with torch.cuda.graph(step):
        y2, saved = layer.forward_train(x, w)
        dx, dw = layer.backward(saved, dy, w)
    x.copy_(normal(tokens, k, seed=5))
    dy.copy_(normal(tokens, n, seed=6))
    forward.replay()
    step.replay()
    y, s = layer.forward_train(x, w)
    want = layer.backward(s, dy, w)
    assert torch.equal(y, y1) and torch.equal(y, y2) and torch.equal(dx, want[0]) and torch.equal(dw, want[1])
    layer.check()


def test_another_stream_and_batched_shapes():
    layer = tsp.TSPLinearE4M3(60, 256, 128)
    w = layer.quantize_weight(normal(256, 128, seed=1))
    x = normal(3, 20, 128, seed=2).bfloat16()
    want = layer.forward(x, w)
    assert want.shape == (3, 20, 256)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = layer.forward(x, w, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_layers_on_two_streams_at_once():
    """An object each: their calls overlap."""
    tokens, n, k = 300, 1000, 2000
    x, dy = normal(tokens, k, seed=2).bfloat16(), normal(tokens, n, seed=3).bfloat16()
    layers = [tsp.TSPLinearE4M3(tokens, n, k) for _ in range(2)]
    w = layers[0].quantize_weight(0.05 * normal(n, k, seed=1))
    y, saved = layers[0].forward_train(x, w)
    want = (y, *layers[0].backward(saved, dy, w))
    for layer in layers:
        layer.enable_backward()
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for layer, s, out in zip(layers, streams, got):
            y, saved = layer.forward_train(x, w, stream=s)
            out.append((y, *layer.backward(saved, dy, w, stream=s)))
    torch.cuda.synchronize()
    for out in got:
        for result in out:
            assert all(torch.equal(a, b) for a, b in zip(result, want))
        del out[:]
    for layer in layers:
        layer.check()


def test_a_layer_refuses_what_does_not_fit():
    layer = tsp.TSPLinearE4M3(10, 64, 48)
    w = layer.quantize_weight(normal(64, 48, seed=1))
    x, dy = normal(6, 48, seed=2).bfloat16(), normal(6, 64, seed=3).bfloat16()
    _, saved = layer.forward_train(x, w)
    out = torch.empty(6, 64, device="cuda")
    x8 = torch.zeros(6, 40, dtype=torch.uint8, device="cuda").view(E4M3)
    for match, call in [
            ("made for 10", lambda: layer.forward(normal(11, 48, seed=2).bfloat16(), w)),
            ("shape", lambda: layer.forward(x[:, :40].contiguous(), w)),
            ("bfloat16", lambda: layer.forward(x.float(), w)),
            ("out must be", lambda: layer.forward(x, w, out=out)),
            ("weight must have shape", lambda: layer.forward(x, tsp.TSPLinearE4M3(1, 48, 64).quantize_weight(normal(48, 64, seed=1)))),
            ("x must have shape", lambda: layer.forward(x8, w, scales=torch.ones(6, 1, device="cuda"))),
            ("expected a weight", lambda: layer.quantize_weight(normal(48, 64, seed=1))),
            ("transpose", lambda: layer.backward(saved, dy, w[:2])),
            ("saved belongs", lambda: layer.backward(saved, dy[:5].contiguous(), w)),
            ("saved belongs", lambda: layer.backward((saved[0][:-1], 6), dy, w)),
            ("needs a dw", lambda: layer.backward(saved, dy, w, accumulate=True))]:
        with pytest.raises(ValueError, match=match):
            call()


def test_no_tokens():
    layer = tsp.TSPLinearE4M3(10, 64, 32)
    w = layer.quantize_weight(normal(64, 32, seed=1))
    x = torch.empty(0, 32, dtype=torch.bfloat16, device="cuda")
    y, saved = layer.forward_train(x, w)
    dx, dw = layer.backward(saved, y, w)
    assert y.shape == (0, 64) and dx.shape == (0, 32) and bool((dw == 0).all())
