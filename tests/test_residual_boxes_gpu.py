"""Whole tiles with a residual, whose pieces go through a warp's two boxes, followed by a split
tile's partial through the same boxes: an odd number of pieces (a last tile of few columns) and
short K-loops, on two and three CTA pairs that walk many tiles each."""
import pytest
import torch

from ff_util import TYPES, matrix
from test_feed_forward_gpu import check_epilogue, operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("N", [40, 96, 192, 296, 352])
@pytest.mark.parametrize("pairs,tiles", [(2, 5), (3, 7), (3, 8)])
@pytest.mark.parametrize("K", [64, 128, 520])
def test_partial_after_residual_tiles(N, pairs, tiles, K, out):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    h = g.Gemm(0)
    h.set_option("cta_pair", 2)
    h.set_option("stream_k", 2)
    h.set_option("max_ctas", 2 * pairs)
    M = 256 * tiles - 56
    a, b = operands(M, N, K, "bf16", 3)
    r = matrix(M, N, TYPES[out], 6)
    first = check_epilogue(h, a, b, None, None, r, out_dtype=out, save=False)
    for _ in range(20):
        assert torch.equal(h.matmul_epilogue(a, b, residual=r, out_dtype=out), first)
    assert h.status() == 0
    h.close()
