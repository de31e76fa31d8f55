"""The objects around the operators on the host: which device they take, which one they launch
on, and what their workspaces do when they grow. No GPU: what allocates or launches is replaced."""
import torch

import pytest

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
operators = tsp.operators


@pytest.fixture
def second_device(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)


@pytest.mark.parametrize("device, want", [(None, 1), (0, 0), (1, 1), ("cuda:0", 0), ("cuda", 1),
                                          (torch.device("cuda", 0), 0), (torch.device("cuda"), 1)], ids=str)
def test_the_device_asked_for(second_device, device, want):
    assert operators._device(device) == torch.device("cuda", want)


@pytest.mark.parametrize("device", ["cpu", torch.device("cpu"), "meta"], ids=str)
def test_only_cuda_devices(second_device, device):
    with pytest.raises(ValueError, match="CUDA device"):
        operators._device(device)
