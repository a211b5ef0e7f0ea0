"""Handle options and tuned choices hold for the feed-forward operators: a product alone is
gemm_run_ex's, bit for bit, where they steer that; the tensor cores run where they are asked for;
and the CTA cap bounds the persistent kernel."""
import pytest
import torch

from ff_util import TYPES, matrix
from test_feed_forward_gpu import check_epilogue, check_epilogue_backward, check_gated, operands

pytestmark = pytest.mark.gpu


@pytest.fixture()
def h():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    hh = g.Gemm(0)
    yield hh
    assert hh.status() == 0
    hh.close()


SHAPES = [(1, 512, 1024), (3, 264, 1000), (40, 512, 2048), (200, 304, 256)]


@pytest.mark.parametrize("option,value", [("force_path", 1), ("force_path", 2), ("block_n", 128),
                                          ("cta_pair", 1), ("cta_pair", 2), ("max_ctas", 8),
                                          ("force_staging", 1), ("stream_k", 2)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_alone(h, M, N, K, dtype, option, value):
    a, b = operands(M, N, K, dtype, 3)
    h.set_option(option, value)
    got = h.matmul_epilogue(a, b, out_dtype="f32")
    assert torch.equal(got, h.matmul(a, b, out_dtype="f32"))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_tuned_product_and_gradient(h, M, N, K, dtype):
    t = TYPES[dtype]
    a, b = operands(M, N, K, dtype, 3)
    h.tune(a, b, out_dtype="f32", iters=2)
    assert torch.equal(h.matmul_epilogue(a, b, out_dtype="f32"), h.matmul(a, b, out_dtype="f32"))
    dy = matrix(M, N, t, 4)
    h.tune(dy, b.t(), iters=2)
    da = h.matmul_epilogue_backward(dy, a, b, need=(True, False, False))[0]
    assert torch.equal(da, h.matmul(dy, b.t()))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_tensor_cores_where_they_are_asked_for(h, M, N, K):
    """fp32: the tensor cores' product, to which a bias of zeros adds nothing."""
    a, b = operands(M, N, K, "f32", 3)
    zero = torch.zeros(N, device="cuda")
    h.set_option("force_path", 1)
    assert torch.equal(h.matmul_epilogue(a, b, bias=zero), h.matmul(a, b))
    g, u = h.gated(a, b, b, save=True)[1:]
    assert torch.equal(g, h.matmul(a, b)) and torch.equal(u, g)
    check_epilogue(h, a, b, "gelu", zero + 1, matrix(M, N, torch.float32, 5))
    check_epilogue_backward(h, matrix(M, N, torch.float32, 4), a, b, matrix(M, N, torch.float32, 6), "silu")


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (4, 264, 1000)])
def test_tensor_cores_for_few_16_bit_tokens(h, M, N, K):
    """The few-token kernel, which GEMM_OPT_CTA_PAIR 1 names too."""
    a, b = operands(M, N, K, "bf16", 3)
    bias = matrix(1, N, torch.float32, 5)[0]
    h.set_option("force_path", 1)
    got = h.matmul_epilogue(a, b, bias=bias, out_dtype="f32"), *h.gated(a, b, b, save=True)
    h.set_option("force_path", 0)
    h.set_option("cta_pair", 1)
    want = h.matmul_epilogue(a, b, bias=bias, out_dtype="f32"), *h.gated(a, b, b, save=True)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("max_ctas", [1, 2, 3])
def test_cta_cap_of_the_persistent_kernel(h, max_ctas):
    """One pair of CTAs has every tile to itself: no split along K, whatever STREAM_K asks for, and
    so the bits of the unsplit sum."""
    a, b = operands(300, 520, 4096, "bf16", 3)
    bias = matrix(1, 520, torch.float32, 5)[0]
    h.set_option("cta_pair", 2)
    call = lambda: (h.matmul_epilogue(a, b, bias=bias, out_dtype="f32"), *h.gated(a, b, b, save=True))
    h.set_option("stream_k", 1)
    want = call()
    h.set_option("stream_k", 2)
    assert not torch.equal(call()[0], want[0])  # (split over all clusters, the sum's order differs)
    h.set_option("max_ctas", max_ctas)
    assert all(torch.equal(p, q) for p, q in zip(call(), want))
    for cap in (5, 17):
        h.set_option("max_ctas", cap)
        check_epilogue(h, a, b, "silu", bias, matrix(300, 520, torch.bfloat16, 6))
        check_gated(h, a, b, b, "silu", save=True)
