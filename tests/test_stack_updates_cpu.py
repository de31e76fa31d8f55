"""TSPStack's AdamW steps on the host: what a refused step leaves, seeds, masters. No GPU: what allocates or
launches is replaced, the library's checks run."""
from types import SimpleNamespace

import pytest
import torch

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
B = tsp._binding
operators, stack_module = tsp.operators, tsp.stack


@pytest.fixture
def host(monkeypatch):
    """CPU tensors pass for those of device 0; launches are listed by name."""
    import os
    if not os.path.exists(B.library_path()):
        import __graft_entry__
        __graft_entry__.build()
    launched = []

    class Device:
        def __init__(self, device):
            pass

        def __enter__(self):
            pass

        def __exit__(self, *exc):
            pass

    def get_device(t):
        if t is None:
            raise TypeError  # as the method itself does
        return 0

    device = SimpleNamespace(index=0)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(torch.Tensor, "get_device", get_device)
    monkeypatch.setattr(torch.Tensor, "device", device)
    monkeypatch.setattr(operators, "_device", lambda d: device)
    for module in (operators, stack_module):
        monkeypatch.setattr(module, "_not_in_a_capture", lambda *a: None)
    monkeypatch.setattr(operators, "_ready", lambda d: None)
    zeros = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k))
    monkeypatch.setattr(B, "_launch", lambda name, *args: launched.append(name))
    return SimpleNamespace(launched=launched, device=device)


def made(host, **kw):
    stack = object.__new__(tsp.TSPStack)
    stack.device = host.device
    stack.wpack = [torch.randn(300).bfloat16(), torch.randn(257).bfloat16()]
    stack.norms = [torch.ones(64).bfloat16() for _ in range(5)]
    stack.clipper = SimpleNamespace(norm=lambda grads: torch.ones(()))
    stack.masters = stack.optimizers = None
    stack.enable_updates(**kw)
    return stack


def gradients(stack):
    return [torch.ones(p.numel()) for p in stack.wpack + stack.norms]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("wrong", ["short", "long", "a norm's size", "a norm's type", "over a norm's master", "a norm itself",
                                   "max_norm", "a matrix's size"])
def test_a_refused_step_steps_nothing(host, wrong, bits):
    stack = made(host, state_bits=bits)
    grads, kw = gradients(stack), {}
    n = len(stack.wpack)
    if wrong == "short":
        grads = grads[:-1]
    elif wrong == "long":
        grads.append(torch.ones(64))
    elif wrong == "a norm's size":
        grads[n + 1] = torch.ones(63)
    elif wrong == "a norm's type":
        grads[-1] = torch.ones(64, dtype=torch.float64)
    elif wrong == "over a norm's master":
        grads[-1] = stack.masters[1][-1]
    elif wrong == "a norm itself":
        grads[-1] = stack.norms[-1]
    elif wrong == "max_norm":
        kw["max_norm"] = -1.0
    else:
        grads[0] = torch.ones(301)
    with pytest.raises((ValueError, B.TSPError)):
        stack.step(grads, 1e-3, **kw)
    assert host.launched == []
    assert [o.t for o in stack.optimizers] == [0, 0]


def test_a_step_steps_both_lists(host):
    stack = made(host)
    stack.step(gradients(stack), 1e-3, max_norm=1.0)
    assert host.launched == ["tsp_adamw_step"] * 2 and [o.t for o in stack.optimizers] == [1, 1]


@pytest.mark.parametrize("seed", [0, 5, (1 << 32) - 1, -3])
def test_the_lists_random_bits_do_not_meet(host, seed):
    """A step's key goes by seed + t in 32 bits: the two lists' are 2^31 apart, so that no step of one has the key of a
    step of the other."""
    a, b = made(host, seed=seed).optimizers
    assert a.seed & 0xFFFFFFFF == seed & 0xFFFFFFFF
    assert (a.seed - b.seed) & 0xFFFFFFFF == 1 << 31


def test_updates_enabled_again_keep_what_the_masters_hold(host):
    """States begin anew, the masters do not: they hold more than the bfloat16 weights. A weight that has been written
    since is its master's new value."""
    stack = made(host, seed=1)
    masters = [m for ms in stack.masters for m in ms]
    with torch.no_grad():
        for m in masters:
            m.mul_(1 + 2.0 ** -12)  # less than half a step of bfloat16
    for p, m in zip(stack.wpack + stack.norms, masters):
        p.copy_(m)
    stack.wpack[1][7:9] = 3.0
    stack.norms[2].fill_(0.5)
    want = [m.clone() for m in masters]
    want[1][7:9], want[len(stack.wpack) + 2][:] = 3.0, 0.5
    stack.step(gradients(stack), 1e-3)
    stack.enable_updates(seed=2, state_bits=8)
    again = [m for ms in stack.masters for m in ms]
    assert all(torch.equal(a, b) for a, b in zip(again, want)) and all(a is b for a, b in zip(again, masters))
    assert [o.t for o in stack.optimizers] == [0, 0] and [o.state_bits for o in stack.optimizers] == [8, 8]
    assert all(a is b for o, ms in zip(stack.optimizers, stack.masters) for a, b in zip(o.masters, ms))


def test_updates_are_not_enabled_in_a_capture(host, monkeypatch):
    stack = made(host)
    before = stack.masters, stack.optimizers

    def capturing(device, what):
        raise RuntimeError(f"{what} cannot be captured")
    monkeypatch.setattr(stack_module, "_not_in_a_capture", capturing)
    monkeypatch.setattr(torch, "where", lambda *a: pytest.fail("work before the refusal"))
    with pytest.raises(RuntimeError, match="enable_updates"):
        stack.enable_updates()
    assert stack.masters is before[0] and stack.optimizers is before[1]
