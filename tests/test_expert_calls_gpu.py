"""Calls of the operators of experts that their documentation allows and no other test makes."""
import pytest
import torch

from expert_util import make_ids, sort_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    return g


@pytest.fixture()
def h(g):
    handle = g.Gemm(0)
    yield handle
    assert handle.status() == 0
    handle.close()


@pytest.mark.parametrize("tokens,k", [(100, 3), (150000, 2), (300000, 2)])  # 4, 8 and 16 ids a lane
@pytest.mark.parametrize("experts", [681, 682, 683])
def test_sort_around_48_kb(h, tokens, k, experts):
    """Tables of counts of 48 KB and a little less and more."""
    ids = make_ids(tokens, k, experts, experts, none=0.1)
    position, offsets = h.expert_sort(ids, experts)
    want = sort_reference(ids, experts)
    assert torch.equal(position.cpu(), want[0]) and torch.equal(offsets.cpu(), want[1])
