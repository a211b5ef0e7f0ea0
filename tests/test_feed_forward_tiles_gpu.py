"""The two tensor-core kernels behind the feed-forward operators, each at the sizes where its
tiles, pieces and pipeline begin and end: the CTA-pair kernel (GEMM_OPT_CTA_PAIR = 2) whole
and split along K, and the few-token kernel with its K-loop shared over clusters
(GEMM_OPT_CTA_PAIR = 1); and their bounded waits."""
import pytest
import torch

from ff_util import TYPES, matrix
from test_feed_forward_gpu import (check_epilogue, check_epilogue_backward, check_gated,
                                   check_gated_backward, operands)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    return g


@pytest.fixture(scope="module", params=["pair", "pair_split", "few"])
def h(request, g):
    hh = g.Gemm(0)
    hh.set_option("cta_pair", 1 if request.param == "few" else 2)
    if request.param == "pair_split":
        hh.set_option("stream_k", 2)
    yield hh
    assert hh.status() == 0
    hh.close()


# rows and columns around 32-row slabs, 64-column pieces, 128-row halves, 256-wide tiles
SIZES = [(1, 1, 8), (1, 260, 640), (31, 64, 64), (33, 72, 136), (128, 128, 128), (129, 136, 200),
         (255, 264, 1000), (256, 256, 64), (257, 504, 72), (300, 1025, 520), (520, 257, 4096),
         (640, 776, 2048)]


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_epilogue(h, M, N, K, dtype):
    t = TYPES[dtype]
    a, b = operands(M, N, K, dtype, M + N)
    bias, residual = matrix(1, N, t, 5)[0], matrix(M, N, t, 6)
    check_epilogue(h, a, b, "gelu", bias, residual, save=True)
    check_epilogue(h, a, b, "silu", None, residual, save=False)
    check_epilogue(h, a, b, "none", bias, None, save=False)
    check_epilogue(h, a, b, "gelu_tanh", bias, matrix(M, N, torch.float32, 6), out_dtype="f32",
                   save=M % 2 == 0)


@pytest.mark.parametrize("pad,offset", [(8, 8), (4, 4), (3, 1)])
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("M,N,K", [(3, 136, 200), (300, 328, 136)])
def test_epilogue_layouts(h, M, N, K, layout, pad, offset):
    a, b = operands(M, N, K, "bf16", 31, "row", layout, pad, offset)
    store = torch.full((M, N + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    check_epilogue(h, a, b, "relu", matrix(1, N, torch.float32, 5)[0],
                   matrix(M, N, torch.bfloat16, 6, pad=pad, offset=offset), out=store[:, :N])
    assert (store[:, N:] == 7).all()
    r = matrix(M, N, torch.bfloat16, 6, pad=pad, offset=offset)
    check_epilogue(h, a, b, None, None, r, out=r, save=False)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_gated(h, M, F, K, dtype):
    x, wg = operands(M, F, K, dtype, M + F)
    wu = matrix(K, F, TYPES[dtype], 9, "col", scale=K ** -0.5)
    check_gated(h, x, wg, wu, "silu", save=False)
    check_gated(h, x, wg, wu, "gelu", save=True)


@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 1)])
@pytest.mark.parametrize("M,F,K", [(3, 136, 200), (300, 328, 136)])
def test_gated_row_major_weights(h, M, F, K, pad, offset):
    x, wg = operands(M, F, K, "bf16", 31, "row", "row", pad, offset)
    wu = matrix(K, F, torch.bfloat16, 9, "row", pad, offset, scale=0.1)
    check_gated(h, x, wg, wu, "sigmoid", save=True)


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("M,F,K", [(40, 200, 136), (300, 328, 264), (520, 1000, 72)])
def test_gated_backward(h, M, F, K, layout):
    t = torch.bfloat16
    x, wg = operands(M, F, K, "bf16", 31, "row", layout)
    wu = matrix(K, F, t, 9, layout, scale=0.1)
    check_gated_backward(h, matrix(M, F, t, 4), x, wg, wu, matrix(M, F, t, 5), matrix(M, F, t, 6),
                         "silu")


def test_many_rounds_of_tiles(g):
    """More tiles than cluster slots, so that both accumulators and the raster groups are used
    again and again, with the default choice of kernels and of the split."""
    h = g.Gemm(0)
    M, N, K = 4100, 2600, 264
    a, b = operands(M, N, K, "bf16", 3)
    check_epilogue(h, a, b, "gelu", matrix(1, N, torch.bfloat16, 5)[0], matrix(M, N, torch.bfloat16, 6),
                   save=False)
    wu = matrix(K, N, torch.bfloat16, 9, "col", scale=0.06)
    check_gated(h, a, b, wu, "silu", save=True)
    a, b = operands(2300, 2600, 4160, "bf16", 3)  # 1.3 rounds of long K-loops: split by default
    check_epilogue(h, a, b, None, None, matrix(2300, 2600, torch.bfloat16, 6), save=False)
    check_epilogue_backward(h, matrix(2300, 2600, torch.bfloat16, 4), a, b,
                            matrix(2300, 2600, torch.bfloat16, 5), "silu")
    assert h.status() == 0
    h.close()


@pytest.mark.parametrize("stall", [1, 2, 3, 6, 7])
@pytest.mark.parametrize("cta_pair", [1, 2])
def test_bounded_waits_expire_and_the_next_call_is_right(g, cta_pair, stall):
    """A loader that issues nothing, or stops after some stage fills: the call ends, the status
    word says so, and the handle's next calls are right (also with a residual on its way). (K:
    64 K-blocks, so that a loader has more fills to do even where eight CTAs share them.)"""
    h = g.Gemm(0)
    h.set_option("cta_pair", cta_pair)
    a, b = operands(300, 520, 4096, "bf16", 3)
    r = matrix(300, 520, torch.bfloat16, 6)
    h.set_option("wait_timeout_us", 20000)
    h.set_option("fault_stall_producer", stall)
    h.matmul_epilogue(a, b, residual=r)
    assert h.status() == 6
    h.gated(a, b, b)
    assert h.status() == 6
    h.set_option("fault_stall_producer", 0)
    check_epilogue(h, a, b, None, None, r, save=False)
    check_gated(h, a, b, b, "silu", save=True)
    assert h.status() == 0
    h.close()


@pytest.mark.parametrize("stall", [1, 2, 3, 6, 7])
@pytest.mark.parametrize("cta_pair", [1, 2])
def test_bounded_waits_with_few_fills(g, cta_pair, stall):
    """16 K-blocks: a CTA pair's loader has all of them to fill, so each stall is reached. The
    few-row kernel may share them over eight CTAs, two fills each: a loader that would stop after
    three (stalls 6 and 7) then has nothing left to hold back, and the call has to be right."""
    h = g.Gemm(0)
    h.set_option("cta_pair", cta_pair)
    a, b = operands(300, 520, 1024, "bf16", 3)
    r = matrix(300, 520, torch.bfloat16, 6)
    want = h.matmul_epilogue(a, b, residual=r), h.gated(a, b, b)
    assert h.status() == 0
    reached = cta_pair == 2 or stall < 6
    h.set_option("wait_timeout_us", 20000)
    h.set_option("fault_stall_producer", stall)
    for call, w in ((lambda: h.matmul_epilogue(a, b, residual=r), want[0]),
                    (lambda: h.gated(a, b, b), want[1])):
        got = call()
        status = h.status()
        assert status == 6 or (not reached and status == 0 and torch.equal(got, w))
    h.set_option("fault_stall_producer", 0)
    check_epilogue(h, a, b, None, None, r, save=False)
    check_gated(h, a, b, b, "silu", save=True)
    assert h.status() == 0
    h.close()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (3, 1)])
@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8, 9])
@pytest.mark.parametrize("N,K", [(1, 1), (7, 8), (129, 40), (70, 513), (1030, 1024), (33, 8200)])
def test_token_kernel(g, M, N, K, pad, offset, dtype):
    """One to eight tokens on the default choice of kernels: features and K around a warp's
    steps, aligned and unaligned rows."""
    h = g.Gemm(0)
    t = TYPES[dtype]
    a, b = operands(M, N, K, dtype, M + N, "row", "col", pad, offset)
    bias = matrix(1, N, t, 5)[0]
    check_epilogue(h, a, b, "gelu", bias, matrix(M, N, t, 6, pad=pad, offset=offset))
    r = matrix(M, N, t, 6)
    check_epilogue(h, a, b, None, None, r, out=r, save=False)
    wu = matrix(K, N, t, 9, "col", pad, offset, scale=K ** -0.5)
    check_gated(h, a, b, wu, "silu", save=M % 2 == 0)
    assert h.status() == 0
    h.close()


@pytest.mark.parametrize("x_layout,w_layout", [("row", "col"), ("row", "row"), ("col", "row"),
                                               ("col", "col")])
@pytest.mark.parametrize("M,N,K", [(9, 1, 1), (9, 64, 15), (17, 65, 16), (64, 64, 17), (65, 130, 513),
                                   (127, 129, 100), (130, 33, 1000), (200, 260, 64), (500, 500, 400)])
def test_fp32_tile_kernel(g, M, N, K, x_layout, w_layout):
    """Small exact fp32 products of every layout, around the tiles' and steps' edges, with
    unaligned rows; and their gradients, whose products are small too."""
    h = g.Gemm(0)
    t = torch.float32
    for pad, offset in ((0, 0), (3, 1)):
        a, b = operands(M, N, K, "f32", M + N, x_layout, w_layout, pad, offset)
        r = matrix(M, N, t, 6, pad=pad, offset=offset)
        check_epilogue(h, a, b, "gelu", matrix(1, N, t, 5)[0], r)
        check_epilogue(h, a, b, None, None, r, out=r, save=False)
        pre, dy = matrix(M, N, t, 7, pad=pad), matrix(M, N, t, 8, pad=pad)
        check_epilogue_backward(h, dy, a, b, pre, "silu")
    if x_layout == "row":
        wu = matrix(K, N, t, 9, w_layout, 3, 1, scale=K ** -0.5)
        check_gated(h, a, b, wu, "silu", save=M % 2 == 0)
        check_gated_backward(h, dy, a, b, wu, pre, matrix(M, N, t, 11), "silu")
    assert h.status() == 0
    h.close()


@pytest.mark.parametrize("M", [1, 4, 64])
def test_weights_written_by_the_call_before(g, M):
    """Weights that the previous kernel on the stream writes, with no host wait in between: a
    product that starts under that kernel's end has to read them as written, bit for bit."""
    h = g.Gemm(0)
    x = matrix(M, 1024, torch.bfloat16, 3)
    w, w2 = (torch.zeros(2048, 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    up = [matrix(2048, 64, torch.bfloat16, 10 + i) for i in range(4)]
    across = matrix(64, 1024, torch.bfloat16, 9)
    got = []
    for i in range(12):
        h.matmul_epilogue(up[(i + 1) % 4], across, out=w2)
        h.matmul_epilogue(up[i % 4], across, out=w)
        got.append((h.matmul_epilogue(x, w.t()), h.gated(x, w2.t(), w.t())))
    torch.cuda.synchronize()
    for i in range(4):
        wi = h.matmul_epilogue(up[i], across)
        wj = h.matmul_epilogue(up[(i + 1) % 4], across)
        torch.cuda.synchronize()
        y, z = h.matmul_epilogue(x, wi.t()), h.gated(x, wj.t(), wi.t())
        for k in range(i, 12, 4):
            assert torch.equal(got[k][0], y) and torch.equal(got[k][1], z)
    assert h.status() == 0
    h.close()
