"""The feed-forward example end to end: its gradients against automatic differentiation of
the block in 64 bits, its training, and its single-token form."""
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
        "feed_forward_example", os.path.join(ROOT, "examples", "feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype,tol", [(torch.float32, 2e-5), (torch.bfloat16, 2e-2)])
@pytest.mark.parametrize("tokens,width,hidden", [(1, 64, 256), (40, 136, 328), (300, 256, 640)])
def test_block_against_automatic_differentiation(example, dtype, tol, tokens, width, hidden):
    """Relative 2-norms: fp32 values carry some ten roundings of 2^-24 times the sums' growth;
    bf16 ones five stored intermediates of at most 2^-8 each (their errors mostly cancel in
    the sums)."""
    h = example.g.Gemm(0)
    block = example.FeedForward(width, hidden, h, dtype=dtype, seed=3)
    gen = torch.Generator("cuda").manual_seed(4)
    block.norm_w += 0.1 * torch.randn(width, generator=gen, device="cuda")
    block.norm_b += 0.1 * torch.randn(width, generator=gen, device="cuda")
    x = torch.randn(tokens, width, generator=gen, device="cuda").to(dtype)
    dy = torch.randn(tokens, width, generator=gen, device="cuda").to(dtype)
    y, saved = block.forward_saved(x)
    dx, grads = block.backward(dy, saved)
    xr = x.double().requires_grad_(True)
    ps = [p.double().requires_grad_(True) for p in block.parameters()]
    n = torch.nn.functional.layer_norm(xr, (width,), ps[0], ps[1])
    a = torch.nn.functional.silu(n @ ps[2].t()) * (n @ ps[3].t())
    want = xr + a @ ps[4].t() + ps[5]
    want_grads = torch.autograd.grad(want, [xr] + ps, dy.double())
    for got, ref in zip([y, dx] + grads, (want.detach(),) + want_grads):
        assert got.shape == ref.shape
        assert float((got.double() - ref).norm()) <= tol * float(ref.norm())
    assert h.status() == 0
    h.close()


def test_example_trains_and_generates(example):
    losses, apart, status = example.main(steps=40)
    assert status == 0
    assert losses[-1] < 0.7 * losses[0]
    # the same arithmetic in other tile shapes: a few roundings to bf16 apart
    assert apart <= 1e-2
