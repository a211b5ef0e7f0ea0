"""Warps some of whose lanes have nothing to store -- features past N in the few-token kernel,
rows past M where TMA cannot store -- before they read the accumulator again as a whole."""
import pytest
import torch

from ff_util import TYPES, matrix
from test_feed_forward_gpu import check_epilogue, check_gated, operands

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cta_pair", [1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M", [33, 97, 200, 300])
@pytest.mark.parametrize("N,K", [(31, 64), (129, 64), (1001, 64), (260, 40), (363, 1024)])
def test_ragged(M, N, K, dtype, cta_pair):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    h = g.Gemm(0)
    h.set_option("cta_pair", cta_pair)
    t = TYPES[dtype]
    a, b = operands(M, N, K, dtype, M + N)
    wu = matrix(K, N, t, 9, "col", scale=K ** -0.5)
    store = torch.full((M, N + 3), 7.0, dtype=t, device="cuda")
    check_epilogue(h, a, b, "silu", matrix(1, N, t, 5)[0], matrix(M, N, t, 6), out=store[:, :N])
    assert (store[:, N:] == 7).all()
    check_epilogue(h, a, b, "gelu", None, matrix(M, N, torch.float32, 6), out_dtype="f32", save=False)
    check_gated(h, a, b, wu, "silu", save=N % 2 == 0)
    assert torch.equal(h.matmul(a, b, out=store[:, :N]), h.matmul(a, b)) and (store[:, N:] == 7).all()
    assert h.status() == 0
    h.close()
