"""The order of tokens by expert, rows into it and back, against numpy and 64-bit forms.

Bounds (u: half a spacing of the stored type): a combined row is a chain of k multiply-adds and a
sum, each within 2^-24 of the running magnitude: (k + 2) 2^-24 D; a gradient's row is one product
in fp32; a weight's gradient is a chain of N / 32 multiply-adds at most and a tree of 5 + 8 sums:
(N / 32 + 16) 2^-24 D."""
import pytest
import torch

from expert_util import make_ids, sort_reference
from ff_util import TYPES, assert_within, matrix, rounding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    return g


@pytest.fixture(scope="module")
def h(g):
    handle = g.Gemm(0)
    yield handle
    assert handle.status() == 0
    handle.close()


@pytest.mark.parametrize("tokens,k,experts", [
    (1, 1, 1), (1, 4, 32), (3, 2, 2), (7, 3, 5), (64, 8, 64), (1023, 3, 17), (2048, 1, 1024),
    (2049, 1, 1000), (683, 3, 33), (16384, 4, 64), (40001, 7, 255), (300000, 4, 1024), (5, 40, 3)])
@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
def test_sort(h, tokens, k, experts, dtype):
    ids = make_ids(tokens, k, experts, tokens + k, none=0.1, dtype=dtype)
    position, offsets = h.expert_sort(ids, experts)
    want = sort_reference(ids, experts)
    assert position.dtype == offsets.dtype == torch.int32
    assert torch.equal(position.cpu(), want[0])
    assert torch.equal(offsets.cpu(), want[1])


def test_sort_ids_outside(h):
    """Ids below 0 and from `experts` on, also past 32 bits, are no expert; rows of ids may be
    parts of wider ones."""
    wide = torch.full((50, 7), 3, dtype=torch.int64, device="cuda")
    ids = wide[:, 2:5]
    ids[::2, 0] = 5
    ids[1, 1], ids[2, 2], ids[3, 0], ids[4, 1] = -1, 2 ** 32 + 1, -2 ** 63, 2 ** 63 - 1
    position, offsets = h.expert_sort(ids, 5)
    want = sort_reference(ids, 5)
    assert torch.equal(position.cpu(), want[0]) and torch.equal(offsets.cpu(), want[1])


def test_sort_one_expert_takes_all(h):
    ids = torch.full((5000, 2), 6, dtype=torch.int32, device="cuda")
    position, offsets = h.expert_sort(ids, 9)
    assert torch.equal(position.view(-1).cpu(), torch.arange(10000, dtype=torch.int32))
    assert offsets.tolist() == [0] * 7 + [10000] * 3


def test_sort_nothing(h):
    for shape in ((0, 2), (4, 0)):
        position, offsets = h.expert_sort(torch.empty(shape, dtype=torch.int64, device="cuda"), 6)
        assert tuple(position.shape) == shape and offsets.tolist() == [0] * 7
    position, offsets = h.expert_sort(torch.full((4, 2), -1, device="cuda"), 6)
    assert offsets.tolist() == [0] * 7 and (position == -1).all()


def same_bits(a, b):
    view = torch.int32 if a.dtype == torch.float32 else torch.int16
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


SHAPES = [(1, 4, 32, 2048), (7, 3, 5, 1), (33, 2, 4, 8), (65, 1, 9, 255), (300, 3, 17, 256),
          (129, 2, 8, 264), (1023, 3, 17, 1025), (50, 35, 40, 72)]


@pytest.mark.parametrize("tokens,k,experts,N", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
def test_gather(h, tokens, k, experts, N, dtype, pad, offset):
    t = TYPES[dtype]
    x = matrix(tokens, N, t, 1, pad=pad, offset=offset)
    x[0, 0] = float("nan")
    ids = make_ids(tokens, k, experts, 2, none=0.2)
    position, offsets = h.expert_sort(ids, experts)
    rows = int(offsets[-1])
    out = matrix(tokens * k + 5, N, t, 3, pad=pad, offset=offset)
    want = out.clone()
    flat = position.view(-1).long()
    want[flat[flat >= 0]] = x[(torch.arange(tokens * k, device="cuda") // k)[flat >= 0]]
    got = h.expert_gather(x, position, out=out)
    assert got is out and same_bits(got, want)
    fresh = h.expert_gather(x, position)
    assert fresh.shape == (tokens * k, N) and same_bits(fresh[:rows], want[:rows])


def test_positions_outside_are_passed_over(h):
    """Rows that the caller's matrix does not have are neither written nor read."""
    x = matrix(4, 300, torch.float32, 1)
    position = torch.tensor([[0, 7], [2 ** 31 - 1, 1], [-5, 2], [3, 4]], dtype=torch.int32, device="cuda")
    out = torch.zeros(4, 300, device="cuda")
    h.expert_gather(x, position, out=out)
    assert torch.equal(out, torch.stack([x[0], x[1], x[2], x[3]]))
    w = torch.full((4, 2), float("nan"), device="cuda")
    w[position < 4] = 2.0
    w[position < 0] = float("nan")
    y = h.expert_combine(out, position, w)
    assert torch.equal(y, 2 * torch.stack([out[0], out[1], out[2], out[3]]))
    drows, dw = h.expert_combine_backward(x, out, position, torch.ones_like(w),
                                          out=torch.full_like(out, 7.0))
    assert torch.equal(drows, torch.stack([x[0], x[1], x[2], x[3]]))
    assert (dw[(position < 0) | (position >= 4)] == 0).all() and dw[0, 0] != 0


def pairs(tokens, k, experts, dtype, weights, seed, h, N, pad=0, offset=0, none=0.2):
    ids = make_ids(tokens, k, experts, seed, none=none)
    position, offsets = h.expert_sort(ids, experts)
    rows = matrix(tokens * k, N, TYPES[dtype], seed + 1, pad=pad, offset=offset)
    rows[int(offsets[-1]):] = float("nan")  # no pair's
    w = matrix(tokens, k, TYPES[weights], seed + 2).contiguous() if weights else None
    return position, rows, w


def gathered64(rows, position):
    z = rows[position.long().clamp(min=0)].double()
    return torch.where((position >= 0)[:, :, None], z, torch.zeros_like(z))


@pytest.mark.parametrize("tokens,k,experts,N", SHAPES)
@pytest.mark.parametrize("dtype,weights,out", [
    ("f32", "f32", "f32"), ("f16", "f32", "f16"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"),
    ("f16", None, "f32"), ("bf16", None, "bf16"), ("f32", "f16", "bf16")])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
def test_combine(h, tokens, k, experts, N, dtype, weights, out, pad, offset):
    t = TYPES[out]
    position, rows, w = pairs(tokens, k, experts, dtype, weights, 5, h, N, pad, offset)
    if w is not None:
        w[position < 0] = float("nan")
    z = gathered64(rows, position)
    f = (torch.where(position >= 0, w.double(), torch.zeros_like(position, dtype=torch.float64))
         if w is not None else (position >= 0).double())
    want, D = torch.einsum("tkn,tk->tn", z, f), torch.einsum("tkn,tk->tn", z.abs(), f.abs())
    bound = (k + 2) * 2.0 ** -24
    y = h.expert_combine(rows, position, w, out_dtype=t)
    assert y.dtype == t
    assert_within(y, want, bound * D + rounding(want, t) * (1 + bound), "combine")
    res = matrix(tokens, N, t, 9, pad=pad, offset=offset)
    want, D = want + res.double(), D + res.double().abs()
    bound_res = bound * D + rounding(want, t) * (1 + bound)
    y = h.expert_combine(rows, position, w, residual=res, out_dtype=t)
    assert_within(y, want, bound_res, "combine with a residual")
    y = h.expert_combine(rows, position, w, residual=res, out=res)
    assert y is res
    assert_within(res, want, bound_res, "combine in place")


# enough tokens and long enough rows for copies in bulk: one piece and more, the last one short, and
# many rows a token
LONG = [(7300, 1, 9, 776), (1700, 3, 17, 2056), (1250, 8, 40, 4096), (1300, 4, 64, 2048),
        (3000, 2, 16, 1032), (2500, 5, 8, 3000)]


@pytest.mark.parametrize("tokens,k,experts,N", LONG)
@pytest.mark.parametrize("dtype,weights,out", [
    ("f32", "f32", "f32"), ("f16", "f32", "f16"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"),
    ("f16", None, "f32"), ("bf16", None, "bf16"), ("f32", "f16", "bf16")])
@pytest.mark.parametrize("pad", [0, 8])
def test_combine_long(h, tokens, k, experts, N, dtype, weights, out, pad):
    t = TYPES[out]
    position, rows, w = pairs(tokens, k, experts, dtype, weights, 5, h, N, pad)
    if w is not None:
        w[position < 0] = float("nan")
    position[5] = -1
    position[position == 3] = 2 ** 31 - 1
    res = matrix(tokens, N, t, 9, pad=pad)
    store = torch.full((tokens + 2, N + pad), 7.0, dtype=t, device="cuda")
    y = store[1:-1, :N]
    h.expert_combine(rows, position, w, out=y)
    onto = h.expert_combine(rows, position, w, residual=res, out_dtype=t)
    place = res.clone()
    h.expert_combine(rows, position, w, residual=place, out=place)
    assert same_bits(onto, place)
    assert (store[0] == 7).all() and (store[-1] == 7).all() and (store[:, N:] == 7).all()
    assert (y[5] == 0).all() and torch.equal(onto[5], res[5])
    bound = (k + 2) * 2.0 ** -24
    for i in range(0, tokens, 100):  # few tokens: rows read by loads, in the same order
        part = slice(i, min(i + 100, tokens))
        p, f = position[part], None if w is None else w[part]
        assert same_bits(y[part], h.expert_combine(rows, p, f, out_dtype=t))
        assert same_bits(onto[part], h.expert_combine(rows, p, f, residual=res[part], out_dtype=t))
        if i % 500 == 0:
            has = (p >= 0) & (p < rows.shape[0])
            z = gathered64(rows, torch.where(has, p, torch.full_like(p, -1)))
            f = torch.where(has, f.double(), torch.zeros_like(z[..., 0])) if f is not None else has.double()
            want, D = torch.einsum("tkn,tk->tn", z, f), torch.einsum("tkn,tk->tn", z.abs(), f.abs())
            assert_within(y[part], want, bound * D + rounding(want, t) * (1 + bound), "combine")
            want, D = want + res[part].double(), D + res[part].double().abs()
            assert_within(onto[part], want, bound * D + rounding(want, t) * (1 + bound), "onto a residual")


def test_combine_long_captured(h):
    """A captured call reads positions and weights anew, also on a stream of its own."""
    position, rows, w = pairs(1300, 4, 64, "bf16", "f32", 5, h, 2048)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y = h.expert_combine(rows, position, w)
    torch.cuda.synchronize()
    for seed in (6, 7):
        other, _, f = pairs(1300, 4, 64, "bf16", "f32", seed, h, 2048)
        position.copy_(other)
        w.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        kept = rows.clone()
        assert same_bits(y, h.expert_combine(kept, other, f))


def test_combine_waits_are_bounded(g):
    """Copies that never come end in a status, and the handle works on."""
    hh = g.Gemm(0)
    position, rows, w = pairs(1300, 4, 64, "bf16", "f32", 5, hh, 2048, none=0.0)
    want = hh.expert_combine(rows, position, w)
    hh.set_option("wait_timeout_us", 20000)
    hh.set_option("fault_stall_producer", 1)
    hh.expert_combine(rows, position, w)
    assert hh.status() == 6
    hh.set_option("fault_stall_producer", 0)
    assert same_bits(hh.expert_combine(rows, position, w), want) and hh.status() == 0
    hh.close()


@pytest.mark.parametrize("tokens,k,experts,N", SHAPES + [(9, 2, 8, 8192), (2, 2, 4, 5001)])
@pytest.mark.parametrize("dtype,weights,grad", [
    ("f32", "f32", "f32"), ("f16", "f32", "f16"), ("bf16", "bf16", "bf16"), ("bf16", "f32", "f32")])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_combine_backward(h, tokens, k, experts, N, dtype, weights, grad, pad, offset):
    t = TYPES[dtype]
    position, rows, w = pairs(tokens, k, experts, dtype, weights, 11, h, N, pad, offset)
    dy = matrix(tokens, N, TYPES[grad], 12, pad=pad, offset=offset)
    out = torch.full((tokens * k, N), 3.0, dtype=t, device="cuda")
    drows, dw = h.expert_combine_backward(dy, rows, position, w, out=out)
    flat = position.view(-1)
    want = torch.full((tokens * k, N), 3.0, dtype=torch.float64, device="cuda")
    values = (w.double()[:, :, None] * dy.double()[:, None, :]).reshape(-1, N)
    want[flat[flat >= 0].long()] = values[flat >= 0]
    assert_within(drows, want, 2.0 ** -24 * want.abs() + rounding(want, t) * (1 + 2.0 ** -24), "drows")
    z = gathered64(rows, position)
    want = torch.einsum("tkn,tn->tk", z, dy.double())
    D = torch.einsum("tkn,tn->tk", z.abs(), dy.double().abs())
    bound = (N / 32 + 16) * 2.0 ** -24
    assert dw.dtype == w.dtype
    assert_within(dw, want, bound * D + rounding(want, w.dtype) * (1 + bound), "dweights")
    only = h.expert_combine_backward(dy, rows, position, w, need=(False, True))
    assert only[0] is None and torch.equal(only[1], dw)
    only = h.expert_combine_backward(dy, rows, position, w, need=(True, False))
    live = int((position >= 0).sum())
    assert only[1] is None and torch.equal(only[0][:live], drows[:live])
    # the gradient of a gather is the combination without weights
    dx = h.expert_gather_backward(rows, position)
    want, D = z.sum(1), z.abs().sum(1)
    bound = (k + 2) * 2.0 ** -24
    assert_within(dx, want, bound * D + rounding(want, t) * (1 + bound), "dx of a gather")


def test_gradients_against_differences(h):
    """combine is linear in the rows and in the weights: central differences with steps of 1 are
    exact but for the roundings of the two sums, 2^-22 of their magnitudes."""
    tokens, k, N = 5, 3, 40
    position, rows, w = pairs(tokens, k, 4, "f32", "f32", 21, h, N, none=0.15)
    rows = torch.nan_to_num(rows)
    dy = matrix(tokens, N, torch.float32, 22)
    drows, dw = h.expert_combine_backward(dy, rows, position, w, out=torch.zeros_like(rows))

    def loss(r, v):
        y = h.expert_combine(r, position, v).double()
        return float((y * dy.double()).sum()), float((y.abs() * dy.double().abs()).sum())

    for i, j in ((0, 0), (1, 2), (4, 1), (3, 0)):
        up, down = w.clone(), w.clone()
        up[i, j] += 1
        down[i, j] -= 1
        (a, da), (b, db) = loss(rows, up), loss(rows, down)
        # (the shifted weight is rounded too: 2^-24 of it, times the row)
        assert abs((a - b) / 2 - float(dw[i, j])) <= 2.0 ** -19 * (da + db)
    live = int((position >= 0).sum())
    for r, c in ((0, 0), (live - 1, N - 1), (live // 2, 7)):
        up, down = rows.clone(), rows.clone()
        up[r, c] += 1
        down[r, c] -= 1
        (a, da), (b, db) = loss(up, w), loss(down, w)
        assert abs((a - b) / 2 - float(drows[r, c])) <= 2.0 ** -19 * (da + db)


def test_there_and_back(h):
    """Sort, gather and combine with weights that sum to 1 give the tokens back."""
    x = matrix(1000, 520, torch.float32, 31)
    ids = make_ids(1000, 4, 16, 32)
    position, _ = h.expert_sort(ids, 16)
    w = torch.full((1000, 4), 0.25, device="cuda")
    assert torch.equal(h.expert_combine(h.expert_gather(x, position), position, w), x)


def test_empty(h):
    none = torch.empty(0, 2, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    assert h.expert_gather(x, none).shape == (0, 16)
    assert h.expert_combine(x, none).shape == (0, 16)
    position = torch.empty(3, 0, dtype=torch.int32, device="cuda")
    res = torch.ones(3, 16, device="cuda")
    assert torch.equal(h.expert_combine(x, position, residual=res), res)
    assert (h.expert_combine(x, position) == 0).all()
    drows, dw = h.expert_combine_backward(res, x, position, torch.empty(3, 0, device="cuda"))
    assert drows.shape == (0, 16) and dw.shape == (3, 0)
    narrow = torch.full((3, 2), -1, dtype=torch.int32, device="cuda")
    drows, dw = h.expert_combine_backward(torch.empty(3, 0, device="cuda"), torch.empty(6, 0, device="cuda"),
                                          narrow, torch.ones(3, 2, device="cuda"))
    assert (dw == 0).all()


def test_captured_and_replayed(h):
    """A captured chain follows new ids and rows; the workspace of the sort serves both graphs."""
    a, b = make_ids(9000, 2, 32, 41), make_ids(9000, 2, 32, 42)
    ids, x = a.clone(), matrix(9000, 64, torch.bfloat16, 43)

    def chain():
        position, offsets = h.expert_sort(ids, 32)
        return position, offsets, h.expert_combine(h.expert_gather(x, position), position, residual=x)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                outs = chain()
            graphs.append((graph, outs))
    torch.cuda.synchronize()
    h.expert_sort(make_ids(400000, 4, 1024, 44), 1024)  # outgrows the captured workspace
    for source in (b, a):
        ids.copy_(source)
        for graph, outs in graphs:
            graph.replay()
            torch.cuda.synchronize()
            want = sort_reference(source, 32)
            assert torch.equal(outs[0].cpu(), want[0]) and torch.equal(outs[1].cpu(), want[1])
            assert torch.equal(outs[2], (3 * x.float()).bfloat16())


def test_on_another_stream(h):
    ids, x = make_ids(500, 2, 8, 51), matrix(500, 96, torch.float16, 52)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    position, offsets = h.expert_sort(ids, 8, stream=stream)
    rows = h.expert_gather(x, position, stream=stream)
    y = h.expert_combine(rows, position, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    want = sort_reference(ids, 8)
    assert torch.equal(position.cpu(), want[0])
    assert torch.equal(y, (2 * x.float()).half())


def test_offsets_past_32_bits(h):
    """Rows that start past 2^32 elements: 70000 rows 65536 apart, the last ones used."""
    far = torch.zeros(70000, 65536, dtype=torch.bfloat16, device="cuda")
    x = matrix(3, 64, torch.bfloat16, 61)
    position = torch.tensor([[69999], [66000], [5]], dtype=torch.int32, device="cuda")
    out = far[:, :64]
    h.expert_gather(x, position, out=out)
    assert torch.equal(out[position.view(-1).long()], x) and int((out != 0).any(1).sum()) == 3
    assert torch.equal(h.expert_combine(out, position), x)
    dw = h.expert_combine_backward(x, out, position, torch.ones(3, 1, device="cuda"), need=(False, True))[1]
    assert_within(dw[:, 0], (x.double() ** 2).sum(1), 2.0 ** -19 * (x.double() ** 2).sum(1), "dweights")


def test_refusals(g, h):
    f = torch.float32
    x, position = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int64, device="cuda")
    rows, w = torch.zeros(8, 8, device="cuda"), torch.zeros(4, 2, device="cuda")
    with pytest.raises(TypeError):
        h.expert_sort(ids.float(), 4)
    with pytest.raises(ValueError):
        h.expert_sort(ids, 0)
    with pytest.raises(ValueError):
        h.expert_sort(ids.view(-1), 4)
    with pytest.raises(g.GemmError, match="UNSUPPORTED"):
        h.expert_sort(ids, 1025)
    many = g.lib().gemm_expert_sort(h.handle, 2 ** 26 + 1, 1, 4, ids.data_ptr(), 1, 8, position.data_ptr(),
                                    rows.data_ptr(), None)
    assert g.STATUS[many] == "GEMM_ERR_UNSUPPORTED"  # (nothing is read or written)
    with pytest.raises(TypeError):
        h.expert_gather(x, ids)
    with pytest.raises(ValueError):
        h.expert_gather(x[:3], position)
    with pytest.raises(ValueError):
        h.expert_gather(x, position.t())
    with pytest.raises(TypeError):
        h.expert_gather(x, position, out=rows.half())
    with pytest.raises(ValueError):
        h.expert_gather(x, position, out=rows[:, :7])
    with pytest.raises(g.GemmError, match="INVALID_ARG"):
        h.expert_gather(rows[:4], position, out=rows)
    with pytest.raises(TypeError):
        h.expert_gather(x.double(), position)
    with pytest.raises(ValueError):
        h.expert_combine(rows, position, w[:, :1])
    with pytest.raises(TypeError):
        h.expert_combine(rows, position, w, residual=x.half())
    with pytest.raises(g.GemmError, match="INVALID_ARG"):
        h.expert_combine(rows, position, w, out=rows[:4])
    with pytest.raises(g.GemmError, match="INVALID_ARG"):
        h.expert_combine_backward(x, rows, position, w, out=rows)
    with pytest.raises(ValueError):
        h.expert_combine_backward(x, rows, position, w, need=(True, True, True))
    with pytest.raises(ValueError):
        h.expert_combine_backward(x[:, :7], rows, position, w)
