"""The order in which the products' persistent CTAs take their tiles (csrc/tile_walk.h), compiled for the host."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "folded_tensor_sequence_tsp_gb300", "csrc")

SHIM = """
#include "tile_walk.h"
extern "C" int group(long long m, long long n, long long k, long long rows) { return tsp::walk_group(m, n, k, rows); }
extern "C" void coords(int tile, int num_p, int num_q, int group_p, int* out) {
  tsp::tile_coords(tile, num_p, num_q, group_p, out[0], out[1]);
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    cc = shutil.which("g++")
    if not cc:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("walk")
    src, lib = str(d / "walk.cpp"), str(d / "walk.so")
    with open(src, "w") as fh:
        fh.write(SHIM)
    subprocess.run([cc, "-std=c++17", "-O1", "-fsanitize=undefined", "-fsanitize-undefined-trap-on-error", "-fPIC", "-shared",
                    "-I", CSRC, src, "-o", lib], check=True)
    dll = ctypes.CDLL(lib)
    dll.group.argtypes = [ctypes.c_longlong] * 4
    out = (ctypes.c_int * 2)()

    def coords(tile, num_p, num_q, group):
        dll.coords(tile, num_p, num_q, group, out)
        return out[0], out[1]
    return dll.group, coords


def tiles(n):
    return -(-n // 256)


@pytest.mark.parametrize("m, n, k, most", [(1, 1, 1, 1), (600, 13000, 4096, 3), (8192, 8192, 4096, 1), (16384, 11008, 4096, 1),
                                           (16384, 22016, 4096, 32), (70000, 65536, 1000, 131)])
def test_every_tile_once(walk, m, n, k, most):
    group, coords = walk
    p, q, g = tiles(m), tiles(n), group(m, n, k, 256)
    assert g == most
    seen = {coords(t, p, q, g) for t in range(p * q)}
    assert len(seen) == p * q and all(0 <= a < p and 0 <= b < q for a, b in seen)


# short rows and a long B: group * columns would pass 31 bits, were the group not held to the row tiles there are
@pytest.mark.parametrize("m, n, k", [(256, 33554432, 4), (256, 25165824, 3), (129, 1 << 26, 1), (129, 1 << 30, 1), (300, 1 << 30, 16),
                                     (1000, 1 << 28, 1), (1 << 20, 1 << 24, 3), (1 << 30, 49 << 20, 1), (1 << 30, 256, 1 << 30)])
def test_long_and_narrow_products(walk, m, n, k):
    group, coords = walk
    p, q, g = tiles(m), tiles(n), group(m, n, k, 256)
    assert 1 <= g <= p
    if p * q > 1 << 29:  # a pair of CTAs each: refused by the call
        return
    assert g * q <= p * q < 1 << 31
    rng = random.Random(m + n)
    for t in [0, 1, p * q - 1, p * q // 2] + [rng.randrange(p * q) for _ in range(1000)]:
        a, b = coords(t, p, q, g)
        assert 0 <= a < p and 0 <= b < q
        # back from the tile's place to its number
        first = a // g * g
        assert first * q + b * min(g, p - first) + (a - first) == t
