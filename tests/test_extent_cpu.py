"""Whether two strided matrices share a byte (csrc/extent.h, compiled for the host), against sets of bytes, and the
refusals that go by it."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
B = tsp._binding
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "folded_tensor_sequence_tsp_gb300", "csrc")

SHIM = """
#include "extent.h"
extern "C" int overlap(long long a, long long ra, long long wa, long long sa, long long b, long long rb, long long wb, long long sb) {
  return tsp::overlaps(tsp::extent((void*)a, ra, wa, sa), tsp::extent((void*)b, rb, wb, sb));
}
"""


@pytest.fixture(scope="module")
def overlap(tmp_path_factory):
    cc = shutil.which("g++")
    if not cc:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("extent")
    src, lib = str(d / "extent.cpp"), str(d / "extent.so")
    with open(src, "w") as fh:
        fh.write(SHIM)
    subprocess.run([cc, "-std=c++17", "-O1", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", "-fPIC", "-shared",
                    "-I", CSRC, src, "-o", lib], check=True)
    fn = ctypes.CDLL(lib).overlap
    fn.argtypes = [ctypes.c_longlong] * 8
    return fn


def taken(at, rows, width, stride):
    return {at + i * stride + j for i in range(rows) for j in range(width)}


@pytest.mark.parametrize("kind", ["same stride", "one run", "unlike strides"])
def test_against_sets_of_bytes(overlap, kind):
    rng = random.Random(3)
    found = [0, 0]
    for _ in range(4000):
        wa, wb, ra, rb = rng.randint(0, 9), rng.randint(0, 9), rng.randint(0, 6), rng.randint(0, 6)
        sa = max(wa, 1) + rng.randint(0, 12)
        sb = max(wb, 1) + rng.randint(0, 12)
        if kind == "same stride":
            sa = sb = max(sa, sb)
        elif kind == "one run":
            ra, sa = (1, sa) if rng.random() < 0.5 else (ra, max(wa, 1))
            wa = sa if ra != 1 and wa else wa
        a, b = 1000 + rng.randint(0, 80), 1000 + rng.randint(0, 80)
        want = bool(taken(a, ra, wa, sa) & taken(b, rb, wb, sb))
        for got in (overlap(a, ra, wa, sa, b, rb, wb, sb), overlap(b, rb, wb, sb, a, ra, wa, sa)):
            assert bool(got) == want or (kind == "unlike strides" and got), (a, ra, wa, sa, b, rb, wb, sb)
        found[want] += 1
    assert min(found) > 300


def test_far_ends(overlap):
    """Matrices whose last byte would be behind the address space's end."""
    big = 1 << 40
    between = (1 << 30) - (1 << 24)
    assert overlap(1 << 24, 1 << 30, between, 4 * big, 1 << 30, 1, 16, 16) == 0
    assert overlap(1 << 24, 1 << 30, between + 1, 4 * big, 1 << 30, 1, 16, 16) == 1
    assert overlap(1 << 24, 1 << 30, 1 << 20, big, (1 << 24) + (1 << 20), 1 << 30, 1 << 20, big) == 0
    assert overlap(1 << 24, 1 << 30, (1 << 20) + 1, big, (1 << 24) + (1 << 20), 1 << 30, 1 << 20, big) == 1


# ------------------------------------------------------------------ refusals: nothing is launched

@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return B.load_library()


P = lambda i: 1 << (24 + i)  # noqa: E731


def refused(status):
    return status == B.TSP_ERR_INVALID_ARG and "alias" in B.tsp_last_error()


@pytest.mark.parametrize("block", [1, 128])
def test_the_quantisers_outputs_lie_apart(lib, block):
    def call(x=P(0), y=P(1), s=P(2), yt=P(3), st=P(4)):
        return lib.tsp_quantize_e4m3(200, 300, x, 0, 304, block, y, 304, s, yt, 208, st, None)
    xbytes = (199 * 304 + 300) * 2
    for kw in (dict(y=P(0) + 16), dict(y=P(0) + xbytes - 1), dict(x=P(1) - 300 * 2 + 2), dict(yt=P(1) + 299), dict(s=P(0) + 4),
               dict(st=P(1) + 8), dict(s=P(3) + 299 * 208), dict(st=P(2) + 4), dict(yt=P(0) + 608 * 100)):
        assert refused(call(**kw)), kw


@pytest.mark.parametrize("b_block", [1, 128])
def test_the_products_output_lies_apart(lib, b_block):
    def call(a=P(0), sa=P(1), b=P(2), sb=P(3), c=P(4)):
        return lib.tsp_matmul_e4m3(200, 300, 400, a, 400, sa, b, 416, sb, b_block, c, 304, 0, 0, P(5), None)
    for kw in (dict(c=P(0) + 399), dict(c=P(0) + 199 * 400), dict(c=P(2) + 2), dict(c=P(1) + 4), dict(c=P(3) + 4),
               dict(sa=P(4) + 608 * 199 + 596), dict(b=P(4) + 16), dict(a=P(4) + 608 * 199 + 592)):
        kw = {k: v & ~1 if k == "c" else v for k, v in kw.items()}
        assert refused(call(**kw)), kw
