"""Scales that the packed attention refuses: its kernels work in base 2, so scale log2(e) has to
be finite in fp32 too. Every call here fails its host checks or has nothing to do."""
import numpy as np
import pytest

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
B = tsp._binding

MAX = float(np.finfo(np.float32).max)
LOG2E = np.float32(1.4426950408889634)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(B.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    return B.load_library()


def calls(lib, scale):
    """Forward and backward without a sequence: nothing to do once the scale is accepted."""
    head = (16, 0, None, 4, 2, 64, scale)
    return (lib.tsp_packed_attention_fwd(*head, *(None, 0) * 5, None, None),
            lib.tsp_packed_attention_bwd(*head, *(None, 0) * 9, None, None))


@pytest.mark.parametrize("scale", [MAX, MAX / 1.4, 2.4e38])
def test_scales_that_overflow_in_base_2(lib, scale):
    with np.errstate(over="ignore"):
        assert np.isinf(LOG2E * np.float32(scale))
    for status in calls(lib, scale):
        assert status == B.TSP_ERR_INVALID_ARG and "scale" in B.tsp_last_error()


@pytest.mark.parametrize("scale", [2.3e38, 1.0, 0.125, 1e-38, 1.5e-45])
def test_scales_that_do_not(lib, scale):
    assert np.isfinite(LOG2E * np.float32(scale)) and LOG2E * np.float32(scale) > 0
    assert calls(lib, scale) == (B.TSP_OK, B.TSP_OK)
