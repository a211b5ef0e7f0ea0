"""Tokens of a block split over experts one at a time and few at once, as a generation loop runs them."""
import importlib.util
import os

import pytest
import torch

from ff_util import UNIT

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
@pytest.mark.parametrize("width,hidden,experts,choices", [(64, 128, 4, 1), (136, 328, 5, 3), (256, 640, 16, 2)])
def test_tokens_one_at_a_time(example, dtype, tol, width, hidden, experts, choices):
    """Each call's y against 64 bits, for the experts that the call itself chose. Relative 2-norms: the
    block's own part as in test_block_against_automatic_differentiation, and the rounding of y, which
    is mostly its residual."""
    h = example.g.Gemm(0)
    block = example.ExpertFeedForward(width, hidden, experts, choices, h, dtype=dtype, seed=3)
    x = torch.randn(24, width, generator=torch.Generator("cuda").manual_seed(4), device="cuda").to(dtype)
    for first, last in [(i, i + 1) for i in range(8)] + [(8, 10), (10, 24)]:
        part = x[first:last].clone()
        ids, _ = block.route(h.layer_norm(part, block.norm_w, block.norm_b))
        want = block.reference(part, torch.zeros_like(part), ids)[0]
        bound = tol * (want - part.double()).norm() + UNIT[dtype] * want.norm()
        y = block.forward(part)
        assert float((y.double() - want).norm()) <= float(bound)
        assert block.forward(part, out=part) is part and torch.equal(part, y)
    assert h.status() == 0
    h.close()
