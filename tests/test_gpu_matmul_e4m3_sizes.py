"""tsp_matmul_e4m3 at the ends of its sizes."""
import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def ws():
    t = torch.zeros(tsp.tsp_matmul_e4m3_workspace_bytes(), dtype=torch.uint8, device="cuda")
    yield t
    assert tsp.tsp_device_status(t) == tsp.TSP_OK


@pytest.mark.parametrize("m, n, pad, dtype", [(1, (1 << 29) + 5, 0, torch.float32), (3, 11, 1 << 29, torch.float32),
                                              (2, 1 << 30, 0, torch.bfloat16), (500, 300, 20, torch.float32), (1, 1, 0, torch.bfloat16)])
def test_an_empty_sum_over_long_rows(m, n, pad, dtype, ws):
    """k 0 gives zeros, also where c's rows are 2^31 bytes apart and more; what lies behind a row stays."""
    c = torch.full((m, n + pad), 3.0, dtype=dtype, device="cuda")
    a, b = (torch.empty(r, 0, dtype=E4M3, device="cuda") for r in (m, n))
    sa, sb = torch.empty(m, 0, device="cuda"), torch.empty(-(-n // 128), 0, device="cuda")
    tsp.tsp_matmul_e4m3(a, sa, b, sb, c[:, :n], ws)
    assert bool((c[:, :n] == 0).all()) and bool((c[:, n:] == 3).all())


def operand(rows, k, seed, block):
    """(e4m3 [rows, k] in rows of a multiple of 16 bytes, scales): whole numbers of -8 to 8 and powers of two, so that a
    sum of few terms is exact."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    up, blocks = -(-k // 16) * 16, -(-k // 128)
    x = torch.empty(rows, up, dtype=torch.uint8, device="cuda").view(E4M3)
    for i in range(0, rows, 1 << 24):
        part = x[i:i + (1 << 24)]
        part.copy_(torch.randint(-8, 9, part.shape, generator=g, device="cuda", dtype=torch.int8).half())
    return x[:, :k], 2.0 ** torch.randint(-3, 4, (-(-rows // block), blocks), generator=g, device="cuda")


# outputs of more than 2^31 elements: by TMA, row by row, and by the kernel for few rows; a long and narrow b, whose
# tiles are walked in one group of all its rows
@pytest.mark.parametrize("m, n, k, dtype", [(70000, 40000, 16, torch.bfloat16), (70001, 40001, 7, torch.bfloat16),
                                            (100, 1 << 25, 16, torch.bfloat16), (256, 25165824, 3, torch.bfloat16),
                                            (300, 9000001, 5, torch.float32)])
def test_outputs_beyond_32_bits(m, n, k, dtype, ws):
    a, sa = operand(m, k, 1, 1)
    b, sb = operand(n, k, 2, 128)
    c = torch.empty(m, n, dtype=dtype, device="cuda")
    tsp.tsp_matmul_e4m3(a, sa, b, sb, c, ws)
    x, wide = a.float() * sa, sb.repeat_interleave(128, 0)[:n]
    step = 1 << 22
    for r in range(0, m, 1000):  # sums of at most 16 products of 8 bits: exact in fp32 whatever the order
        for s in range(0, n, step):
            y = b[s:s + step].float() * wide[s:s + step]
            want = x[r:r + 1000] @ y.t() if k > 1 else x[r:r + 1000] * y.t()
            assert torch.equal(c[r:r + 1000, s:s + step], want.to(dtype)), (r, s)
