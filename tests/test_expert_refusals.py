"""The module's functions of experts and dropout refuse operands in host memory, and operands that
are no tensors, also where there is no GPU."""
import pytest
import torch

import dense_tiled_gemm_05_gb300 as g

X, IDS = torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64)
POSITION, W = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
W3, OFFSETS = torch.zeros(3, 8, 6), torch.zeros(4, dtype=torch.int32)

CALLS = {
    "expert_sort": lambda x: g.expert_sort(x, 4),
    "expert_gather": lambda x: g.expert_gather(x, POSITION),
    "expert_gather_backward": lambda x: g.expert_gather_backward(x, POSITION),
    "expert_combine": lambda x: g.expert_combine(x, POSITION, W),
    "expert_combine_backward": lambda x: g.expert_combine_backward(x, X, POSITION, W),
    "expert_matmul": lambda x: g.expert_matmul(x, W3, OFFSETS),
    "expert_matmul_backward": lambda x: g.expert_matmul_backward(x, X, W3, OFFSETS),
    "expert_gated": lambda x: g.expert_gated(x, W3, W3, OFFSETS),
    "expert_gated_backward": lambda x: g.expert_gated_backward(x, X, W3, W3, X, X, OFFSETS),
    "dropout": lambda x: g.dropout(x, 0.5, torch.zeros(2, dtype=torch.int64)),
    "dropout_backward": lambda x: g.dropout_backward(x, 0.5, torch.zeros(2, dtype=torch.int64)),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_host_tensors(name):
    with pytest.raises(ValueError, match="CUDA tensors"):
        CALLS[name](IDS if name == "expert_sort" else X)


@pytest.mark.parametrize("name", list(CALLS))
def test_no_tensors(name):
    with pytest.raises(TypeError):
        CALLS[name]([[1.0, 2.0]])


def test_null_handles():
    """The C entries check their arguments before anything else."""
    L = g.lib()
    assert L.gemm_expert_sort(None, 1, 1, 1, None, 1, 8, None, None, None) == 1
    assert L.gemm_expert_gather(None, 1, 1, 1, None, 1, None, 1, None, 1, 0, None) == 1
    assert L.gemm_expert_combine(None, 1, 1, 1, None, 1, 1, None, None, 0, None, 1, None, 1, 0, 0, None) == 1
    assert L.gemm_expert_combine_backward(None, 1, 1, 1, None, 1, None, 1, 1, None, None, 0, None, 1, None,
                                          0, 0, None) == 1
    assert L.gemm_run_expert(None, 1, 1, 1, 1, None, 1, None, 1, 1, None, None, 1, 2, 1, None) == 1
    assert L.gemm_run_expert_backward(None, 1, 1, 1, 1, None, 1, None, 1, None, 1, 1, None, None, 1, None,
                                      1, 1, 2, 1, None) == 1
    assert L.gemm_run_expert_gated(None, 1, 1, 1, 1, None, 1, None, 1, 1, None, 1, 1, None, None, 1, None,
                                   1, None, 1, 2, 1, 4, None) == 1
    assert L.gemm_run_expert_gated_backward(None, 1, 1, 1, 1, None, 1, None, 1, None, 1, None, 1, None, 1,
                                            1, None, 1, 1, None, None, 1, None, 1, 1, None, 1, 1, 2, 1, 4,
                                            None) == 1
    assert L.gemm_dropout(None, 1, 1, None, 1, None, 1, None, 1, 0.5, None, 0, None) == 1
