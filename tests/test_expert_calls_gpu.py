"""Calls of the operators of experts that their documentation allows and no other test makes."""
import pytest
import torch

from expert_util import make_ids, sort_reference
from ff_util import acc_error, assert_within, matrix, rounding
from test_expert_products_gpu import offsets_of

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


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


def test_surplus_rows_after_many_whole_blocks(g):
    """A weight gradient whose only ragged expert comes after some 50 tiles a cluster of one without
    surplus rows: the warp that clears surplus rows waits longer than any single step takes, and the
    limit of a wait is still one step's. (1024 rows of 16384 x 16384: 330 us in all, 6 us a tile.)"""
    hh = g.Gemm(0)
    offsets, bounds = offsets_of([1024, 1003])
    x, dy = matrix(bounds[-1], 16384, BF16, 1), matrix(bounds[-1], 16384, BF16, 2)
    w = torch.empty(2, 16384, 16384, dtype=BF16, device="cuda").transpose(1, 2)
    want = hh.expert_matmul_backward(dy, x, w, offsets, need=(False, True))[1]
    assert hh.status() == 0
    hh.set_option("wait_timeout_us", 100)
    for _ in range(3):
        got = hh.expert_matmul_backward(dy, x, w, offsets, need=(False, True))[1]
        assert hh.status() == 0
        assert torch.equal(got, want)
    a, b = bounds[1], bounds[2]
    xd, d = x[a:b, :300].double(), dy[a:b, -300:].double()
    ref, D = xd.t() @ d, xd.abs().t() @ d.abs()
    assert_within(got[1][:300, -300:], ref, 1.01 * acc_error(BF16, b - a) * D + rounding(ref, BF16), "dw")
    hh.close()
