"""GPU: the example layer trains, decodes in four bits, and can be captured with its gradients into a graph."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("moe_layer", os.path.join(ROOT, "examples", "moe_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_it_trains_and_decodes(example):
    losses, off = example.run()
    assert losses[-1] < losses[0], losses
    # a code is off by up to half a step of (max - min) / 15, evenly spread: 1 / sqrt(12) of a step, and a group of 64
    # normal values spans some 4.6 deviations, so a weight is off by 0.09 of its deviation. Two products and the gated
    # activation between them (three factors) add up to about twice that.
    assert 0 < off < 0.3, off


def test_quantized_weights_are_within_half_a_step(example):
    w = torch.randn(2, 24, 128, device="cuda").bfloat16()
    q, scale, zero = example.quantize(w)
    code = torch.stack([q & 15, q >> 4], -1).flatten(-2).float()
    back = (code - zero.float().repeat_interleave(64, -1)) * scale.float().repeat_interleave(64, -1)
    # half a step for the code and half for the zero point, and the scale's own rounding over 15 steps
    assert bool(((back - w.float()).abs() <= scale.float().repeat_interleave(64, -1) * (1 + 15 * 2.0 ** -8)).all())


def test_forward_and_backward_in_a_graph(example):
    """No eager graph of the same leaves is alive at the capture; replays, eager work between, equal eager steps."""
    moe = example.moe
    T, H, W, E, k = 200, 64, 96, 4, 2
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    x, w_in, w_out, dout = normal(T, H), normal(E, 2 * W, H) / 8, normal(E, H, W) / 8, normal(T, H)
    router = torch.randn(H, E, generator=g, device="cuda")
    for t in (x, w_in, w_out):
        t.requires_grad_(True)

    def step():
        out = example.layer(x, router, w_in, w_out, k, lambda r, w, o: moe.grouped_matmul(r, w, o, layout="nk"))
        return (out.detach(),) + torch.autograd.grad(out, (x, w_in, w_out), dout)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for i in range(4):
        with torch.no_grad():
            x.copy_(normal(T, H))
            dout.copy_(normal(T, H))
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(a, b), i
