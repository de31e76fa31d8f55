"""The quantiser and the AdamW step on matrices and tensors of more than 2^31 elements: the same bits as calls on parts."""
import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def bytes_(x):
    return x.view(torch.uint8)


@pytest.mark.parametrize("rows, width, block", [(70016, 40000, 1), (70001, 40003, 1), (70001, 40003, 128), (33, 1 << 27, 1)])
def test_quantising_beyond_32_bits(rows, width, block):
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    blocks, up = lambda n: -(-n // 128), lambda n: -(-n // 16) * 16  # noqa: E731
    of = lambda r, w: torch.empty(r if block == 1 else blocks(r), blocks(w), device="cuda")  # noqa: E731
    y, s = torch.empty(rows, up(width), dtype=E4M3, device="cuda")[:, :width], of(rows, width)
    yt, st = torch.empty(width, up(rows), dtype=E4M3, device="cuda")[:, :rows], of(width, rows)
    tsp.tsp_quantize_e4m3(x, y, s, yt, st, block=block)
    # the corners: the last rows and columns, and the middle, each of them where blocks begin
    for r in {0, rows // 256 * 128, (rows - 1) // 128 * 128}:
        for c in {0, width // 256 * 128, (width - 1) // 128 * 128 - 128}:
            part = x[r:r + 128, c:c + 1000].contiguous()
            n, w = part.shape
            y1, s1 = torch.empty(n, up(w), dtype=E4M3, device="cuda")[:, :w], of(n, w)
            yt1, st1 = torch.empty(w, up(n), dtype=E4M3, device="cuda")[:, :n], of(w, n)
            tsp.tsp_quantize_e4m3(part, y1, s1, yt1, st1, block=block)
            rb, cb = (r, c) if block == 1 else (r // 128, c // 128)
            whole = w // 128 * 128 if c + w < width else w  # a block that the part cuts has another scale
            k, kb = whole, blocks(whole)
            assert torch.equal(bytes_(y[r:r + n, c:c + k]), bytes_(y1[:, :k])), (r, c)
            assert torch.equal(s[rb:rb + s1.shape[0], c // 128:c // 128 + kb], s1[:, :kb])
            assert torch.equal(bytes_(yt[c:c + k, r:r + n]), bytes_(yt1[:k])), (r, c)
            kt = k if block == 1 else kb
            assert torch.equal(st[cb:cb + kt, r // 128:r // 128 + 1], st1[:kt])


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_beyond_32_bits(bits):
    """From zero states a step does not depend on the states' bits: every part moves as in a call of its own."""
    n = (1 << 31) + 4096 * 5 + 77
    g = torch.Generator(device="cuda").manual_seed(6)
    p, grad = (torch.empty(n, device="cuda").normal_(generator=g) for _ in range(2))
    ends = [(0, 5000), ((1 << 31) - 3000, (1 << 31) + 3000), (n - 5000, n)]
    parts = [(p[a:b].clone(), grad[a:b].clone()) for a, b in ends]
    opt = tsp.TSPAdamW([p], state_bits=bits)
    opt.step([grad], 1e-3)
    for (a, b), (q, d) in zip(ends, parts):
        own = tsp.TSPAdamW([q])
        own.step([d], 1e-3)
        assert torch.equal(p[a:b], q)
        if bits == 32:
            assert torch.equal(opt.m[0][a:b], own.m[0]) and torch.equal(opt.v[0][a:b], own.v[0])
        else:
            for state, scales, want in ((opt.m, opt.m_scales, own.m[0]), (opt.v, opt.v_scales, own.v[0])):
                s = scales[0][a // 128:-(-b // 128)].repeat_interleave(128)[a % 128:a % 128 + b - a]
                got = state[0][a:b].float() * s
                # a neighbour: within a step, 2^-3 of the value or 2^-9 of the scale, and 16 of the bits it is chosen by
                assert bool(((got - want).abs() <= (want.abs() * 2.0 ** -3).clamp_min(2.0 ** -9 * s) * 1.0001).all())
