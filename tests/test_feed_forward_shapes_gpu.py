"""Operands of one row or one column, cut from wider buffers: their strides allow both layouts,
and the gradients' buffers must be written in the one that the call names."""
import pytest
import torch

from ff_util import TYPES, matrix
from test_feed_forward_gpu import check_epilogue, check_epilogue_backward, check_gated, check_gated_backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    hh = g.Gemm(0)
    yield hh
    assert hh.status() == 0
    hh.close()


def column(n, t, seed, wide=3):
    """A 1 x n view with stride (1, wide): one column of an n x wide buffer, transposed."""
    return matrix(n, wide, t, seed)[:, 1:2].t()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("K", [1, 5, 200, 1024])
@pytest.mark.parametrize("b_layout", ["row", "col"])
def test_one_row_from_a_column(h, K, b_layout, dtype):
    t = TYPES[dtype]
    a, b = column(K, t, 1), matrix(K, 40, t, 2, b_layout, scale=K ** -0.5)
    assert a.stride() == (1, 3)
    check_epilogue(h, a, b, "silu", None, matrix(1, 40, t, 3))
    check_epilogue_backward(h, matrix(1, 40, t, 4), a, b, matrix(1, 40, t, 5), "silu")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 40), (7, 5), (200, 264)])
@pytest.mark.parametrize("a_layout", ["row", "col"])
def test_one_input_with_a_column_for_its_weights(h, M, N, a_layout, dtype):
    t = TYPES[dtype]
    a, b = matrix(M, 1, t, 1, a_layout), column(N, t, 2)
    check_epilogue(h, a, b, "gelu", None, None)
    check_epilogue_backward(h, matrix(M, N, t, 4), a, b, matrix(M, N, t, 5), "gelu")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("need", [(True, True, True), (False, True, False), (False, False, True)])
@pytest.mark.parametrize("M,F", [(1, 40), (33, 72)])
def test_gated_pair_of_one_input(h, M, F, need, dtype):
    t = TYPES[dtype]
    x, wg, wu = matrix(M, 1, t, 1), column(F, t, 2), column(F, t, 3, wide=4)
    check_gated(h, x, wg, wu, "silu", save=True)
    check_gated_backward(h, matrix(M, F, t, 4), x, wg, wu, matrix(M, F, t, 5), matrix(M, F, t, 6),
                         "silu", need)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_single_rows_and_columns_of_any_stride(h, dtype):
    """X[:1, ::3] is a row, W[::2, :1] a column: each reads as a matrix of one line."""
    t = TYPES[dtype]
    a, b = matrix(4, 300, t, 1)[2:3, ::3], matrix(100, 40, t, 2, "col", scale=0.1)
    assert a.shape == (1, 100) and a.stride() == (300, 3)
    check_epilogue(h, a, b, "silu", None, None)
    check_epilogue_backward(h, matrix(1, 40, t, 4), a, b, matrix(1, 40, t, 5), "silu")
    a, b = matrix(9, 100, t, 1), matrix(200, 5, t, 2, scale=0.1)[::2, 1:2]
    assert b.shape == (100, 1)
    check_epilogue(h, a, b, "silu", None, None)
    check_epilogue_backward(h, matrix(9, 1, t, 4), a, b, matrix(9, 1, t, 5), "silu")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("swap", [False, True])
def test_gated_weights_of_one_row_or_column(h, swap, dtype):
    """One weight tight, the other cut from a wider buffer: both have a common layout."""
    t = TYPES[dtype]
    for K, F, wg, wu in ((1, 40, matrix(1, 40, t, 2), column(40, t, 3)),
                         (24, 1, matrix(24, 1, t, 2, "col"), matrix(24, 3, t, 3)[:, 1:2])):
        x, wg, wu = matrix(7, K, t, 1), *((wu, wg) if swap else (wg, wu))
        check_gated(h, x, wg, wu, "silu", save=True)
        check_gated_backward(h, matrix(7, F, t, 4), x, wg, wu, matrix(7, F, t, 5), matrix(7, F, t, 6), "silu")
