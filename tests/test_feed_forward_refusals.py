"""The module's feed-forward functions refuse operands in host memory, and operands that are no
tensors, as the handle's methods do -- also where there is no GPU."""
import pytest
import torch

import dense_tiled_gemm_05_gb300 as g

X, W, V = torch.zeros(4, 8), torch.zeros(8, 6), torch.zeros(4)

CALLS = {
    "matmul_epilogue": lambda x: g.matmul_epilogue(x, W),
    "matmul_epilogue_backward": lambda x: g.matmul_epilogue_backward(torch.zeros(4, 6), x, W),
    "gated": lambda x: g.gated(x, W, W),
    "gated_backward": lambda x: g.gated_backward(torch.zeros(4, 6), x, W, W, torch.zeros(4, 6),
                                                 torch.zeros(4, 6)),
    "layer_norm": lambda x: g.layer_norm(x),
    "layer_norm_backward": lambda x: g.layer_norm_backward(X, x, None, V, V),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_host_tensors(name):
    with pytest.raises(ValueError, match="CUDA tensors"):
        CALLS[name](X)


@pytest.mark.parametrize("name", list(CALLS))
def test_no_tensors(name):
    with pytest.raises(TypeError):
        CALLS[name]([[1.0, 2.0]])
