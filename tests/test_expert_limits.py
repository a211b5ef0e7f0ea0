"""Sizes at the limits of the operators of experts: the C entries take them or refuse them before they
read the handle or launch anything, so that no operand of such a size is needed (nor a GPU). A size
that is taken shows in the next check, of a pointer that is not aligned."""
import ctypes

import pytest

import dense_tiled_gemm_05_gb300 as g

INT32_MAX = 2 ** 31 - 1
F32, BF16, ROW, SILU = 0, 2, 0, 4
OK, UNSUPPORTED, ALIGNMENT = 0, 2, 3
HANDLE = ctypes.create_string_buffer(4096)  # never read
P, ODD = 4096, 4099  # addresses that nothing reads


def product(rows, N, K, dtype):
    return g.lib().gemm_run_expert(HANDLE, 1, rows, N, K, P, K, P, N, K * N, ODD, P, N, dtype, ROW, None)


def product_backward(rows, N, K, dtype):
    return g.lib().gemm_run_expert_backward(HANDLE, 1, rows, N, K, P, N, P, K, P, N, K * N, ODD, P, K, P, N,
                                            K * N, dtype, ROW, None)


def gated(rows, N, K, dtype):
    return g.lib().gemm_run_expert_gated(HANDLE, 1, rows, N, K, P, K, P, N, K * N, P, N, K * N, ODD, P, N,
                                         None, 0, None, 0, dtype, ROW, SILU, None)


def gated_backward(rows, N, K, dtype):
    return g.lib().gemm_run_expert_gated_backward(
        HANDLE, 1, rows, N, K, P, N, P, N, P, N, P, K, P, N, K * N, P, N, K * N, ODD, P, K, P, N, K * N, P, N,
        K * N, dtype, ROW, SILU, None)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("call", [product, product_backward, gated, gated_backward])
def test_products(call, dtype):
    """Rows are counted in tiles of up to 256 and features in tiles of 256, in 32 bits: a size is
    refused where rounding it up leaves them."""
    most = INT32_MAX - 511
    for rows, N, K in ((most, 8, 8), (1, 8, most)):
        assert call(rows, N, K, dtype) == ALIGNMENT
    for size in (most + 1, INT32_MAX - 255, INT32_MAX - 62, INT32_MAX, INT32_MAX + 1):
        assert call(size, 8, 8, dtype) == UNSUPPORTED
        assert call(1, 8, size, dtype) == UNSUPPORTED
        assert call(1, size, 8, dtype) == UNSUPPORTED


def gather(tokens, k):
    return g.lib().gemm_expert_gather(HANDLE, tokens, k, 8, P, 8, ODD, 4, P, 8, BF16, None)


def combine(tokens, k):
    return g.lib().gemm_expert_combine(HANDLE, tokens, k, 8, P, 8, 4, ODD, None, F32, None, 0, P, 8, BF16,
                                       BF16, None)


def combine_backward(tokens, k):
    return g.lib().gemm_expert_combine_backward(HANDLE, tokens, k, 8, P, 8, P, 8, 4, ODD, None, F32, P, 8, None,
                                                BF16, BF16, None)


@pytest.mark.parametrize("call", [gather, combine, combine_backward])
def test_choices(call):
    """A warp takes a token's pairs 32 at a time, in 32 bits: a last step past INT32_MAX is refused."""
    assert call(1, INT32_MAX - 31) == ALIGNMENT
    assert call(INT32_MAX, 1) == ALIGNMENT
    for k in (INT32_MAX - 30, INT32_MAX, INT32_MAX + 1):
        assert call(1, k) == UNSUPPORTED
    assert call(2 ** 16, 2 ** 15) == UNSUPPORTED
