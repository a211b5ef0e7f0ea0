"""The block split over experts end to end: its gradients against automatic differentiation in 64
bits, its training loop and single tokens, and a captured step."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    spec = importlib.util.spec_from_file_location(
        "expert_feed_forward_example", os.path.join(ROOT, "examples", "expert_feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype,tol", [(torch.float16, 4e-3), (torch.bfloat16, 3e-2)])
@pytest.mark.parametrize("tokens,width,hidden,experts,choices,drop", [
    (1, 64, 128, 4, 1, 0.0), (40, 136, 328, 5, 3, 0.3), (300, 256, 640, 16, 2, 0.1), (700, 200, 72, 3, 2, 0.5)])
def test_block_against_automatic_differentiation(example, dtype, tol, tokens, width, hidden, experts,
                                                 choices, drop):
    """Relative 2-norms: some eight stored intermediates, each rounded by at most half a step (2^-8
    bf16, 2^-11 f16), whose errors mostly cancel in the sums: sqrt(8) half steps and as much again
    for the products they enter twice."""
    h = example.g.Gemm(0)
    block = example.ExpertFeedForward(width, hidden, experts, choices, h, drop=drop, dtype=dtype, seed=3)
    gen = torch.Generator("cuda").manual_seed(4)
    block.norm_w += 0.1 * torch.randn(width, generator=gen, device="cuda")
    block.norm_b += 0.1 * torch.randn(width, generator=gen, device="cuda")
    x = torch.randn(tokens, width, generator=gen, device="cuda").to(dtype)
    dy = torch.randn(tokens, width, generator=gen, device="cuda").to(dtype)
    y, saved = block.forward_saved(x)
    dx, grads = block.backward(dy, saved)
    for got, ref in zip([y, dx] + grads, block.reference(x, dy, saved[4])):
        assert got.shape == ref.shape
        # (with one choice a token its weight is 1: the router has no gradient)
        assert float((got.double() - ref).norm()) <= tol * float(ref.norm()) + 1e-12
    assert h.status() == 0
    h.close()


def test_example_runs(example):
    losses, apart, status = example.main(steps=3)
    assert status == 0
    assert all(v == v and v < float("inf") for v in losses + [apart])


def test_captured_step(example):
    """A step captured in a graph and replayed with other tokens, whose experts get other numbers of
    rows, and with the next dropout mask, gives what an eager step gives."""
    h = example.g.Gemm(0)
    block = example.ExpertFeedForward(128, 96, 6, 2, h, drop=0.2, seed=5)
    gen = torch.Generator("cuda").manual_seed(6)
    xs = [torch.randn(150, 128, generator=gen, device="cuda").bfloat16() for _ in range(3)]
    dy = torch.randn(150, 128, generator=gen, device="cuda").bfloat16()
    x = xs[0].clone()

    def step():
        y, saved = block.forward_saved(x)
        return [y] + [v for part in block.backward(dy, saved) for v in (part if isinstance(part, list) else [part])]

    step()  # (grows the handle's buffers)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        outs = step()
    torch.cuda.synchronize()
    for i, source in enumerate(xs):
        x.copy_(source)
        block.key[1] = i
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
    assert h.status() == 0
    h.close()
