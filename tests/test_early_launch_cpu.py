"""Kernels that launch_early starts while the kernel before them is still writing: none of their
pointers may be declared read-only for the kernel's lifetime (const with __restrict__), which
would let the compiler load through the non-coherent path or before the wait."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "folded_tensor_sequence_tsp_gb300", "csrc")


def sources():
    out = {}
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        with open(path) as fh:
            text = re.sub(r"//[^\n]*", "", fh.read())
        out[os.path.basename(path)] = text
    return out


def early(text):
    """Names of the kernels that a file hands to launch_early, through a local `kernel` or not."""
    names = set()
    for m in re.finditer(r"launch_early\(\s*(\w+)", text):
        name = m.group(1)
        if name == "kernel":  # the nearest definition above
            name = re.findall(r"auto kernel = (\w+)", text[:m.start()])[-1]
        names.add(name)
    return names


def parameters(text, kernel):
    m = re.search(r"__global__[^;{]*?\b" + kernel + r"\((.*?)\)\s*\{", text, flags=re.S)
    return m.group(1) if m else None


def test_no_early_kernel_declares_what_it_reads_read_only():
    found = 0
    for name, text in sources().items():
        for kernel in early(text):
            params = parameters(text, kernel)
            assert params is not None, (name, kernel)
            assert not re.search(r"\bconst\b[^,]*__restrict__", params), (name, kernel)
            found += 1
    assert found >= 5  # list readers of both attentions' sides, dw's sum, norm's join, scaling


@pytest.mark.parametrize("what", ["partial", "items", "short_count", "count"])
def test_what_the_earlier_kernel_leaves_is_not_loaded_through_ldg(what):
    for name, text in sources().items():
        assert not re.search(r"__ldg\([^;]*\b" + what + r"\b", text), name
