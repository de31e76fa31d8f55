"""TSPStack and the packed attention's object beside captures: a graph of the forward that was
captured before the stack grew its workspace, and objects made inside a capture."""
import pytest
import torch

import gpu_util as gu
import tsp_inputs

tsp = pytest.importorskip("folded_tensor_sequence_tsp_gb300")
pytestmark = pytest.mark.gpu

NAMES = ("Wq", "Wk", "Wv", "Wo", "W1", "W3", "W2")


def make(S=256):
    cfg = tsp_inputs.LayerConfig("t", 2, S, 256, 4, 688, 3)
    b = tsp_inputs.layer_inputs(cfg)
    w = {k: gu.dev(b[k]) for k in NAMES}
    w["attn_norm"] = w["mlp_norm"] = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    return tsp.TSPStack(2, S, 256, 4, 688, [w], w["attn_norm"]), gu.dev(b["x"])


def capture(call):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = call()
    torch.cuda.current_stream().wait_stream(side)
    return graph, out


def test_a_forward_graph_outlives_the_growth_of_the_workspace():
    stack, xs = make()
    want = stack.forward(xs).clone()
    graph, out = capture(lambda: stack.forward(xs))
    small = stack.ws.numel()
    trained, saved = stack.forward_train(xs)
    assert stack.ws.numel() > small and torch.equal(trained, want)
    # memory of the old workspace's size, if it had been given back
    others = [torch.full((small,), 0x5a, dtype=torch.uint8, device="cuda") for _ in range(4)]
    for _ in range(2):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want)
    assert all(bool((t == 0x5a).all()) for t in others)
    stack.check()


def test_constructors_and_growth_refuse_a_capture():
    stack, xs = make()
    stack.forward(xs)
    torch.cuda.synchronize()

    def inside():
        with pytest.raises(RuntimeError, match="before the capture"):
            tsp.TSPPackedAttention(64, 2, 4, 2, 64)
        with pytest.raises(RuntimeError, match="before the capture"):
            stack.forward_train(xs)
        return stack.forward(xs)  # needs nothing of the kind

    want = stack.forward(xs).clone()
    graph, out = capture(inside)
    graph.replay()
    assert torch.equal(out, want)
    stack.check()
