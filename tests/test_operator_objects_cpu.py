"""The objects around the operators on the host: which device they take, which one they launch
on, and what their workspaces do when they grow. No GPU: what allocates or launches is replaced."""
import gc
import weakref
from types import SimpleNamespace

import pytest
import torch

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


# ------------------------------------------------------------------ TSPStack
stack_module = tsp.stack


class Fakes:
    """The calls of a TSPStack as records of (name, device current at the call)."""

    def __init__(self, monkeypatch):
        self.calls, self.current = [], None
        fakes = self

        class Device:
            def __init__(self, device):
                self.device = device

            def __enter__(self):
                self.before, fakes.current = fakes.current, self.device

            def __exit__(self, *exc):
                fakes.current = self.before

        def record(name, result=None):
            def call(*args, **kwargs):
                fakes.calls.append((name, fakes.current))
                return result
            return call

        info = SimpleNamespace(D=2, T=4, batch=1, hidden=8, tokens=8, wpack_elems=16)
        monkeypatch.setattr(torch.cuda, "device", Device)
        monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: self.capturing)
        monkeypatch.setattr(torch.cuda, "current_stream",
                            lambda device=None: SimpleNamespace(cuda_stream=0, synchronize=record("synchronize")))
        self.capturing = False
        monkeypatch.setattr(stack_module, "_device", lambda device: torch.device("cpu"))
        for name, result in (("tsp_plan", SimpleNamespace(info=info)), ("tsp_packed_weight_bytes", 32),
                             ("tsp_workspace_bytes", 256), ("tsp_bwd_workspace_bytes", 512),
                             ("tsp_workspace_init", None), ("tsp_pack_weights", None),
                             ("tsp_attention_fwd", None), ("tsp_mlp_fwd", None), ("tsp_attention_bwd", None),
                             ("tsp_mlp_bwd", None), ("tsp_device_status", 0)):
            monkeypatch.setattr(stack_module, name, record(name, result))

        class Norm:
            def __init__(self, *args, **kwargs):
                pass

            def forward(self, x, w, residual=None, y=None, h=None):
                return x.clone(), residual

            def backward(self, h, w, dy, dh=None, dx=None, dx16=None):
                return h.clone(), torch.zeros(8)

        class Clip:
            def __init__(self, *args, **kwargs):
                pass

            def clip(self, grads, max_norm):
                return record("clip")()

        monkeypatch.setattr(stack_module, "TSPRMSNorm", Norm)
        monkeypatch.setattr(stack_module, "TSPGradClip", Clip)

    def stack(self, weights=None):
        if weights is None:
            weights = [{k: torch.zeros(8) for k in ("Wq", "Wk", "Wv", "Wo", "W1", "W3", "W2", "attn_norm",
                                                     "mlp_norm")} for _ in range(2)]
        return tsp.TSPStack(2, 8, 8, 2, 16, weights, torch.zeros(8))


def test_a_stack_launches_on_its_own_device(monkeypatch):
    fakes = Fakes(monkeypatch)
    s = fakes.stack()
    x = torch.zeros(2, 4, 8, dtype=torch.bfloat16)
    s.forward(x)
    out, saved = s.forward_train(x)
    _, grads = s.backward(saved, out)
    s.clip(grads, 1.0)
    s.check()
    launched = {name for name, _ in fakes.calls}
    assert {"tsp_pack_weights", "tsp_workspace_init", "tsp_attention_fwd", "tsp_mlp_fwd", "tsp_attention_bwd",
            "tsp_mlp_bwd", "tsp_device_status", "clip"} <= launched
    for name, device in fakes.calls:
        if name not in ("tsp_plan", "tsp_packed_weight_bytes", "tsp_workspace_bytes", "tsp_bwd_workspace_bytes"):
            assert device == s.device, name
    assert fakes.current is None


def test_a_stack_refuses_weights_of_another_device(monkeypatch):
    fakes = Fakes(monkeypatch)
    w = {k: torch.zeros(8) for k in ("Wq", "Wk", "Wv", "Wo", "W1", "W3", "W2", "attn_norm", "mlp_norm")}
    w["mlp_norm"] = torch.zeros(8, device="meta")
    with pytest.raises(ValueError, match="must be on"):
        fakes.stack([w])


def waits_last(fakes):
    """The last thing that was queued has been waited for, on the right device."""
    name, device = fakes.calls[-1]
    return name == "synchronize" and device == torch.device("cpu")


def test_a_workspace_is_ready_when_the_constructor_returns(monkeypatch):
    """Memory that the constructor took over may still be written by what its stream has queued,
    and the first call may come on another stream."""
    fakes = Fakes(monkeypatch)
    monkeypatch.setattr(operators, "_device", lambda device: torch.device("cpu"))
    for name in ("tsp_packed_attention_workspace_bytes", "tsp_rmsnorm_workspace_bytes", "tsp_grad_workspace_bytes"):
        monkeypatch.setattr(operators, name, lambda *args: 256)
    monkeypatch.setattr(operators, "tsp_status_init", lambda ws: fakes.calls.append(("init", fakes.current)))
    for make in (lambda: tsp.TSPPackedAttention(8, 1, 2, 1, 64), lambda: tsp.TSPRMSNorm(8, 64),
                 lambda: tsp.TSPGradClip(3), fakes.stack):
        fakes.calls.clear()
        make()
        assert waits_last(fakes)
    stack = fakes.stack()
    fakes.calls.clear()
    stack.enable_backward()
    assert waits_last(fakes) and ("tsp_workspace_init", stack.device) in fakes.calls
    fakes.calls.clear()
    stack.enable_backward()  # nothing to grow
    assert all(name == "tsp_bwd_workspace_bytes" for name, _ in fakes.calls)


def test_what_zeroes_a_status_word_is_not_captured(monkeypatch):
    """Inside a capture the zeroing would wait for a replay, and a call outside it would find
    counters of any value."""
    fakes = Fakes(monkeypatch)
    monkeypatch.setattr(operators, "_device", lambda device: torch.device("cpu"))
    stack = fakes.stack()
    fakes.capturing = True
    before = stack.ws
    fakes.calls.clear()
    x = torch.zeros(2, 4, 8, dtype=torch.bfloat16)
    for call in (lambda: tsp.TSPPackedAttention(8, 1, 2, 1, 64), fakes.stack, stack.enable_backward,
                 lambda: stack.forward_train(x)):
        with pytest.raises(RuntimeError, match="before the capture"):
            call()
    assert stack.ws is before and all(name == "tsp_bwd_workspace_bytes" for name, _ in fakes.calls)
    stack.forward(x)  # needs nothing of the kind
    fakes.capturing = False
    stack.enable_backward()
    fakes.capturing = True
    stack.forward_train(x)


def test_a_graph_keeps_the_workspace_it_was_captured_with(monkeypatch):
    """forward_train grows the workspace; a graph of the forward, captured earlier, writes to the
    one before it when it is replayed."""
    stack = Fakes(monkeypatch).stack()
    captured = weakref.ref(stack.ws)
    stack.forward_train(torch.zeros(2, 4, 8, dtype=torch.bfloat16))
    gc.collect()
    assert stack.ws.numel() == 512 and captured() is not None
    looked_at = []
    monkeypatch.setattr(stack_module, "tsp_device_status", lambda ws: looked_at.append(ws.numel()) or 0)
    stack.check()
    assert sorted(looked_at) == [256, 512]
    del stack
    gc.collect()
    assert captured() is None
