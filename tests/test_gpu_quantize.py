"""tsp_quantize_e4m3 bit for bit against its definition: scales are fp32 quotients of the block's
largest magnitude by 448, values fp32 quotients by the scale rounded to e4m3 (a quotient in 64 bits of
fp32 numbers, rounded to fp32, is the fp32 quotient: 53 bits are more than twice 24 and two)."""
import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def blocks(n):
    return -(-n // 128)


def reference(x, block):
    """(codes as bytes, scales) of a matrix on the CPU, a scale for 128 columns of one or 128 rows."""
    x = x.double()
    rows, w = x.shape
    codes = torch.zeros(rows, w, dtype=torch.uint8)
    scales = torch.zeros(-(-rows // block), blocks(w))
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            part = x[i * block:(i + 1) * block, 128 * j:128 * (j + 1)]
            top = part.abs().max()  # a NaN stays one
            s = torch.tensor(1.0) if top == 0 else (top / 448).float().clamp_min(2.0 ** -126)
            scales[i, j] = s
            q = (part / s.double()).float().clamp(-448, 448).to(E4M3)
            codes[i * block:(i + 1) * block, 128 * j:128 * (j + 1)] = q.view(torch.uint8)
    return codes, scales


def outputs(rows, w, block, ld_y, ld_yt):
    dev = dict(device="cuda")
    y = torch.full((rows, ld_y), 0xA5, dtype=torch.uint8, **dev)
    yt = torch.full((w, ld_yt), 0xA5, dtype=torch.uint8, **dev)
    s = torch.full((-(-rows // block), blocks(w)), -1.0, **dev)
    st = torch.full((-(-w // block), blocks(rows)), -1.0, **dev)
    return y, s, yt, st


def check(x, block, which="both", pad=0, base=0):
    """x on the GPU; pad: elements behind the rows of y and yt, which have to stay as they were."""
    rows, w = x.shape
    y, s, yt, st = outputs(rows, w, block, w + pad, rows + pad)
    args = {}
    if which != "transpose":
        args |= dict(y=y.view(E4M3)[:, :w], scales=s)
    if which != "rows":
        args |= dict(yt=yt.view(E4M3)[:, :rows], scales_t=st)
    tsp.tsp_quantize_e4m3(x, block=block, **args)
    xc = x.cpu()
    if which != "transpose":
        codes, scales = reference(xc, block)
        assert torch.equal(s.cpu(), scales)
        assert torch.equal(y[:, :w].cpu(), codes)
    if which != "rows":
        codes, scales = reference(xc.t(), block) if block == 1 else [t.t() for t in reference(xc, block)]
        assert torch.equal(st.cpu(), scales)
        assert torch.equal(yt[:, :rows].cpu(), codes)
    assert bool((y[:, w:] == 0xA5).all()) and bool((yt[:, rows:] == 0xA5).all())


def draw(rows, w, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, w, generator=g) * torch.exp(2 * torch.randn(w, generator=g))
    return x.to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("which", ["both", "rows", "transpose"])
@pytest.mark.parametrize("rows, w, pad", [(1, 1, 0), (3, 127, 1), (128, 128, 0), (129, 260, 12), (5, 1024, 16),
                                          (300, 100, 0), (144, 16, 0)])
def test_forms(dtype, block, which, rows, w, pad):
    check(draw(rows, w, dtype, rows * w + pad), block, which, pad)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("first, last", [(0, 256), (4, 132), (1, 130), (8, 264)])
def test_column_ranges_of_a_wider_matrix(dtype, block, first, last):
    check(draw(140, 300, dtype, 5)[:, first:last], block, pad=4)


@pytest.mark.parametrize("block", [1, 128])
def test_special_blocks(block):
    x = torch.randn(256, 384, generator=torch.Generator().manual_seed(9))
    x[:128, :128] = 0
    x[5, 3] = -0.0
    x[:128, 128:256] *= 1e-42           # subnormal: the smallest scale holds
    x[128:, :128] *= 1e37
    x[130, 7] = 3.4028234663852886e38   # the largest number
    x[128:, 256:] = x[128:, 256:].bfloat16().float().clamp(-3, 3)
    check(x.cuda(), block)


@pytest.mark.parametrize("block", [1, 128])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")], ids=str)
def test_what_is_not_finite_stays_in_its_blocks(block, bad):
    x = torch.randn(256, 256, generator=torch.Generator().manual_seed(11))
    x[3, 5] = bad
    y, s, yt, st = outputs(256, 256, block, 256, 256)
    tsp.tsp_quantize_e4m3(x.cuda(), y.view(E4M3), s, yt.view(E4M3), st, block=block)
    hit = torch.zeros(s.shape, dtype=torch.bool)
    hit[3 // block, 0] = True
    hit_t = torch.zeros(st.shape, dtype=torch.bool)
    hit_t[5 // block, 0] = True
    for got, where in ((s.cpu(), hit), (st.cpu(), hit_t)):
        assert torch.equal(~torch.isfinite(got), where)
    clean = x.clone()
    clean[3, 5] = 0
    codes, _ = reference(clean, block)
    rows = torch.repeat_interleave(torch.repeat_interleave(hit, block, 0), 128, 1)
    assert torch.equal(y.cpu()[~rows], codes[~rows])


@pytest.mark.parametrize("block", [1, 128])
def test_quotients_next_to_ties(block):
    """Scales whose mantissas are within some units of a multiple of 2^19, and values whose quotients by them are
    within some units of halfway between two e4m3 values: where an approximate quotient would round wrongly."""
    g = torch.Generator().manual_seed(3)
    rows = []
    for near in (0, 1, 2, 5, 11, 15, 16, 17, 18, 40):
        for sign in (1, -1):
            for j in (16, 17, 21, 26, 31):
                s = torch.tensor((j << 19) + sign * near, dtype=torch.float64) * 2.0 ** -30
                top = (s * 448).float()
                scale = (top.double() / 448).float().double()  # what the block's largest value makes of it
                # ties: 1.0001 to 1.1111 in binary, and between subnormal values
                t = (2 * torch.randint(8, 16, (63,), generator=g) + 1).double() * 2.0 ** torch.randint(-10, 4, (63,), generator=g)
                t = torch.cat([t, (2 * torch.randint(0, 8, (64,), generator=g) + 1).double() * 2.0 ** -10])
                ulp = 2.0 ** (torch.floor(torch.log2(t)) - 23)
                x = (scale * (t + ulp * torch.randint(-3, 4, (127,), generator=g) / 2)).float()
                bits = x.view(torch.int32) + torch.randint(-1, 2, (127,), generator=g, dtype=torch.int32)
                x = bits.view(torch.float32) * (torch.randint(0, 2, (127,), generator=g) * 2 - 1)
                rows.append(torch.cat([top[None], x]))
    x = torch.stack(rows)
    if block == 1:
        check(x.cuda(), 1)
        check(x.t().contiguous().cuda(), 1)
    else:
        for i in range(0, len(rows), 10):  # one largest value to a tile
            check(x[i:i + 1].repeat(128, 1).cuda(), 128)


def test_empty():
    for rows, w in ((0, 5), (5, 0), (0, 0)):
        x = torch.zeros(rows, w, device="cuda")
        y, s, yt, st = outputs(rows, w, 1, w, rows)
        tsp.tsp_quantize_e4m3(x, y.view(E4M3), s, yt.view(E4M3), st)
