"""Calls of the operators of experts that their documentation allows and no other test makes."""
import pytest
import torch

from expert_util import make_ids, sort_reference
from ff_util import TYPES, acc_error, assert_within, matrix, rounding
from test_expert_products_gpu import offsets_of, weights

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


def backward_into(g, h, counts, layout, place):
    """gemm_run_expert_gated_backward with both weight gradients in one buffer of NaN; place(F, K, E)
    gives (elements, ld, stride, dWu's first element)."""
    offsets, bounds = offsets_of(counts)
    E, K, F, rows = len(counts), 72, 40, bounds[-1]
    x, (dh, gate, up) = matrix(rows, K, BF16, 1), (matrix(rows, F, BF16, s) for s in (2, 3, 4))
    wg, wu = (weights(E, K, F, BF16, s, layout) for s in (5, 6))
    size, ld, stride, second = place(F, K, E)
    buf = torch.full((size,), float("nan"), dtype=BF16, device="cuda")
    lw, sw = (K, F * K) if layout == "col" else (F, F * K)
    p = lambda t: t.data_ptr()
    status = g.lib().gemm_run_expert_gated_backward(
        h.handle, E, rows, F, K, p(dh), F, p(gate), F, p(up), F, p(x), K, p(wg), lw, sw, p(wu), lw, sw,
        p(offsets), None, 0, p(buf), ld, stride, p(buf) + 2 * second, ld, stride, 2,
        1 if layout == "col" else 0, 4, torch.cuda.current_stream().cuda_stream)
    want = h.expert_gated_backward(dh, x, wg, wu, gate, up, offsets, need=(False, True, True))[1:]
    shape = (E, F, K) if layout == "col" else (E, K, F)
    got = [buf[o:].as_strided(shape, (stride, ld, 1)) for o in (0, second)]
    return g.STATUS[status], buf, [v.transpose(1, 2) if layout == "col" else v for v in got], want


# the gradients as column ranges of wider lines (of every expert, or all experts' lines on end), and as
# parts of each expert's block of lines
PLACES = {"columns": lambda F, K, E: (E * K * 2 * F, 2 * F, K * 2 * F, F),
          "columns, gap": lambda F, K, E: (E * (K + 3) * (2 * F + 8), 2 * F + 8, (K + 3) * (2 * F + 8), F + 8),
          "blocks": lambda F, K, E: (E * 2 * K * F, F, 2 * K * F, K * F)}


@pytest.mark.parametrize("place", list(PLACES))
@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("counts", [[90], [5, 0, 70]], ids=str)
def test_weight_gradients_in_one_buffer(g, h, counts, layout, place):
    def at(F, K, E):
        return PLACES[place](F, K, E) if layout == "row" else PLACES[place](K, F, E)
    status, buf, got, want = backward_into(g, h, counts, layout, at)
    assert status == "GEMM_OK"
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    written = sum(v.numel() for v in got)
    assert int(torch.isnan(buf).sum()) == buf.numel() - written


@pytest.mark.parametrize("counts", [[90], [5, 0, 70]], ids=str)
@pytest.mark.parametrize("second", [0, 1, 8, 39])
def test_overlapping_weight_gradients_are_refused(g, h, counts, second):
    """Gradients 40 wide in lines of 80 that start less than 40 apart, and across a line's end."""
    for first in (second, 80 - second):
        status, buf, *_ = backward_into(
            g, h, counts, "row", lambda F, K, E: (E * K * 2 * F + 80, 2 * F, K * 2 * F, first))
        assert status == "GEMM_ERR_INVALID_ARG"
        assert torch.isnan(buf).all()


# rows of a piece and more, the last piece short, for 16-bit and fp32 rows; one choice and many
PIECES = [(1, 776), (2, 1032), (3, 2056), (5, 3000), (8, 1544)]


@pytest.mark.parametrize("k,N", PIECES)
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("onto", [False, True])
def test_combine_by_bulk_copies(g, k, N, dtype, out, onto):
    """Long rows of many tokens come by bulk copies, and have the bits of a few tokens' rows, which come
    by loads. Which of the two a call takes shows when no copy is issued: the waits end in a status."""
    hh = g.Gemm(0)
    tokens = 60 * torch.cuda.get_device_properties(0).multi_processor_count + 5
    position, _ = hh.expert_sort(make_ids(tokens, k, 9, 3, none=0.1), 9)
    rows = matrix(tokens * k, N, TYPES[dtype], 4)
    w = matrix(tokens, k, torch.float32, 5).contiguous()
    t = TYPES[out]
    residual = matrix(tokens, N, t, 6) if onto else None
    y = hh.expert_combine(rows, position, w, residual=residual, out_dtype=t)
    parts = [slice(i, i + 100) for i in range(0, tokens, 100)]

    def few(p):
        return hh.expert_combine(rows, position[p], w[p], residual=residual[p] if onto else None, out_dtype=t)

    for p in parts:
        assert torch.equal(y[p], few(p))
    assert hh.status() == 0
    hh.set_option("wait_timeout_us", 2000)
    hh.set_option("fault_stall_producer", 1)
    few(parts[0])
    assert hh.status() == 0
    hh.expert_combine(rows, position, w, residual=residual, out_dtype=t)
    assert hh.status() == 6
    hh.close()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_first_calls_are_captured(g, dtype):
    """A handle's first calls, captured: its buffers are made, and cleared, outside the graph, and grow
    from one captured call to the next. Replayed twice, with other work between, then called eagerly."""
    t = TYPES[dtype]
    eager, hh = g.Gemm(0), g.Gemm(0)
    ids = make_ids(1500, 2, 6, 7, none=0.1)
    tokens = matrix(1500, 133, t, 1)  # (rows TMA cannot address: copied first)
    wg, wu = (weights(6, 133, 72, t, s) for s in (2, 3))
    w = weights(1, 4096, 256, t, 4)  # few tiles with long K: shared
    x, whole = matrix(5, 4096, t, 5), offsets_of([5])[0]
    dh = matrix(3000, 72, t, 6)
    key = torch.tensor([3, 4], device="cuda")

    def calls(h):
        position, offsets = h.expert_sort(ids, 6)
        rows = h.expert_gather(tokens, position, out=torch.zeros(3000, 133, dtype=t, device="cuda"))
        blank = lambda n: torch.zeros(3000, n, dtype=t, device="cuda")
        y, gate, up = h.expert_gated(rows, wg, wu, offsets, save=True, out=blank(72))
        live = (torch.arange(3000, device="cuda") < offsets[-1]).unsqueeze(1)
        gate, up = (torch.where(live, v, torch.zeros_like(v)) for v in (gate, up))
        return [h.expert_matmul(x, w, whole), position, offsets, rows, y, gate, up,
                *h.expert_gated_backward(dh, rows, wg, wu, gate, up, offsets, out=blank(133)),
                h.dropout(tokens, 0.3, key, residual=tokens)]

    want = calls(eager)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        got = calls(hh)
    torch.cuda.synchronize()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
            a.zero_()
    for a, b in zip(calls(hh), want):
        assert torch.equal(a, b)
    assert hh.status() == 0 and eager.status() == 0
    del graph
    hh.close()
    eager.close()
