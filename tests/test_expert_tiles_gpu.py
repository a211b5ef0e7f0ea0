"""Tiles of the experts' products: shared K, many tiles a row of tiles, options, weights in every
order of memory, elements past 2^31 and 2^32, the same bits again, and workspaces that graphs share."""
import pytest
import torch

from ff_util import TYPES, acc_error, assert_within, matrix, rounding
from test_expert_products_gpu import (check_backward, check_gated, check_gated_backward, check_product,
                                      offsets_of, rows_with_gaps, sentinel, weights)

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
    torch.cuda.empty_cache()


# few tiles with long K (shared by auto), rounds of tiles that end unevenly, narrow and wide tiles
SHARED = [([3], 200, 4096), ([1, 0, 40], 256, 8192), ([600], 300, 4100), ([100, 513, 0, 7], 264, 2048),
          ([300] * 9, 2600, 1024), ([20] * 50, 1000, 1088), ([2600, 300], 520, 200), ([700, 5000], 2560, 136)]


@pytest.mark.parametrize("counts,N,K", SHARED, ids=str)
@pytest.mark.parametrize("stream_k", [0, 1, 2])
@pytest.mark.parametrize("max_ctas", [0, 6])
def test_shared_tiles(h, counts, N, K, stream_k, max_ctas):
    h.set_option("stream_k", stream_k)
    h.set_option("max_ctas", max_ctas)
    offsets, bounds = offsets_of(counts, 1)
    rows = bounds[-1] + 2
    x = rows_with_gaps(rows, K, BF16, 1, bounds)
    w = weights(len(counts), K, N, BF16, 2)
    y = sentinel(rows, N, BF16)
    check_product(h, x, w, offsets, bounds, y)
    again = h.expert_matmul(x, w, offsets)  # the same bits, from a fresh buffer
    assert torch.equal(again[bounds[0]:bounds[-1]], y[bounds[0]:bounds[-1]])
    dy = rows_with_gaps(rows, N, BF16, 3, bounds)
    check_backward(h, dy, x, w, offsets, bounds, sentinel(rows, K, BF16))


@pytest.mark.parametrize("layout", ["col", "row"])
@pytest.mark.parametrize("F", [304, 200])  # interleaved weights, or two accumulators
@pytest.mark.parametrize("counts,K", [([3], 4096), ([600, 9], 2048), ([2600], 264)], ids=str)
@pytest.mark.parametrize("stream_k", [1, 2])
def test_shared_gated_tiles(h, counts, F, K, layout, stream_k):
    h.set_option("stream_k", stream_k)
    offsets, bounds = offsets_of(counts, 1)
    rows = bounds[-1] + 2
    x = rows_with_gaps(rows, K, BF16, 1, bounds)
    wg, wu = (weights(len(counts), K, F, BF16, s, layout) for s in (2, 3))
    check_gated(h, x, wg, wu, offsets, bounds, "silu")
    dh, gate, up = (rows_with_gaps(rows, F, BF16, s, bounds) for s in (4, 5, 6))
    check_gated_backward(h, dh, x, wg, wu, gate, up, offsets, bounds, "silu")


@pytest.mark.parametrize("rows", [5, 400])
def test_gated_weights_in_any_order(h, rows):
    """The gate's weights behind the up projection's, with other expert strides, and one matrix for
    both."""
    offsets, bounds = offsets_of([rows, 0, 33])
    x = matrix(bounds[-1], 128, BF16, 1)
    w = weights(3, 128, 416, BF16, 2)
    check_gated(h, x, w[:, :, 208:], w[:, :, :208], offsets, bounds, "silu")
    check_gated(h, x, w[:, :, :208], w[:, :, 208:], offsets, bounds, "gelu")
    check_gated(h, x, w[:, :, :208], w[:, :, :208], offsets, bounds, "silu")
    check_gated(h, x, weights(3, 128, 208, BF16, 3, gap=64), weights(3, 128, 208, BF16, 4), offsets, bounds, "silu")
    check_gated(h, x, weights(3, 128, 208, BF16, 3, pad=8), weights(3, 128, 208, BF16, 4), offsets, bounds, "silu")


def test_widths_of_tiles(h):
    """Row counts around the steps of 32 and the tiles of 64, 128 and 256 rows, one expert each."""
    counts = [1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 159, 160, 161, 191, 193, 223, 225, 255, 256,
              257, 289, 511, 513, 594, 767, 769]
    offsets, bounds = offsets_of(counts)
    x, w = matrix(bounds[-1], 200, BF16, 1), weights(len(counts), 200, 136, BF16, 2)
    check_product(h, x, w, offsets, bounds, sentinel(bounds[-1], 136, BF16))
    dy = matrix(bounds[-1], 136, BF16, 3)
    check_backward(h, dy, x, w, offsets, bounds, sentinel(bounds[-1], 200, BF16))


def far_rows(rows, cols, t, seed, bounds):
    """Rows whose last ones start more than 2^32 elements into the buffer."""
    ld = -(-(1 << 32) // (rows - 60)) // 8 * 8 + 8
    view = torch.empty((rows - 1) * ld + cols, dtype=t, device="cuda").as_strided((rows, cols), (ld, 1))
    view.copy_(matrix(rows, cols, t, seed))
    return view


@pytest.mark.parametrize("counts", [[90, 0, 43], [2000, 70, 600]], ids=str)
def test_elements_past_32_bits(h, counts):
    """Rows, outputs, kept products and weights more than 2^32 elements from their first."""
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GB")
    offsets, bounds = offsets_of(counts)
    rows, K, N = bounds[-1], 136, 208
    gap = (1 << 31) + 16  # elements between experts
    x = far_rows(rows, K, BF16, 1, bounds)

    def far_weights(seed):
        w = torch.empty(2 * gap + K * N, dtype=BF16, device="cuda").as_strided((3, K, N), (gap, 1, K))
        w.copy_(weights(3, K, N, BF16, seed))
        return w

    w = far_weights(2)
    check_product(h, x, w, offsets, bounds, far_rows(rows, N, BF16, 4, bounds))
    dy = far_rows(rows, N, BF16, 3, bounds)
    out = far_rows(rows, K, BF16, 5, bounds)
    check_backward(h, dy, x, w, offsets, bounds, out)
    del out
    wu = far_weights(6)
    y = h.expert_gated(x, w, wu, offsets, save=True)
    want = h.expert_gated(x.contiguous(), w.contiguous(), wu.contiguous(), offsets, save=True)
    for a, b in zip(y, want):
        assert_within(a, b.double(), 2.0 ** -6 * b.double().abs() + 1e-3, "gated")


def test_many_weights(h):
    """More than 2^32 bytes and 2^31 elements of weights and of their gradients."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    E, N, K = 70, 4096, 7680
    counts = [0] * E
    for e in (0, 34, 68, 69):
        counts[e] = 3 + e
    offsets, bounds = offsets_of(counts)
    w = torch.zeros(E, N, K, dtype=BF16, device="cuda").transpose(1, 2)
    for e in (0, 34, 68, 69):
        w[e] = matrix(K, N, BF16, e, "col", scale=K ** -0.5)
    x, dy = matrix(bounds[-1], K, BF16, 1), matrix(bounds[-1], N, BF16, 2)
    y = h.expert_matmul(x, w, offsets)
    _, dw = h.expert_matmul_backward(dy, x, w, offsets, need=(False, True))
    for e in (0, 34, 68, 69):
        a, b = bounds[e], bounds[e + 1]
        xd, wd, d = x[a:b].double(), w[e].double(), dy[a:b].double()
        want, D = xd @ wd, xd.abs() @ wd.abs()
        assert_within(y[a:b], want, 1.01 * acc_error(BF16, K) * D + rounding(want, BF16), "y of %d" % e)
        want, D = xd.t() @ d, xd.t().abs() @ d.abs()
        assert_within(dw[e], want, 1.01 * acc_error(BF16, b - a) * D + rounding(want, BF16), "dw of %d" % e)
    assert (dw[35:68] == 0).all()


def test_graphs_share_the_workspace(h):
    """Two captured calls whose tiles are shared, wide and narrow ones, replayed in turn between eager
    calls: each reads the epoch and flags of its own launch."""
    wide, narrow = offsets_of([700])[0], offsets_of([4, 0, 9])[0]
    xw, ww = matrix(700, 4096, BF16, 1), weights(1, 4096, 512, BF16, 2)
    xn, wn = matrix(13, 4096, BF16, 3), weights(3, 4096, 256, BF16, 4)
    want = h.expert_matmul(xw, ww, wide), h.expert_matmul(xn, wn, narrow)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        for x, w, o in ((xw, ww, wide), (xn, wn, narrow)):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                outs = h.expert_matmul(x, w, o)
            graphs.append((graph, outs))
    torch.cuda.synchronize()
    for i in range(6):
        for j in (0, 1, 1, 0):
            graph, out = graphs[j]
            out.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[j])
        assert torch.equal(h.expert_matmul(xn, wn, narrow), want[1])
