"""The experts' products on the GPU against their definitions in 64 bits, expert by expert: plain
and gated, with their gradients. Row counts from none to all around every tile's edge, ragged
extents, both layouts, padded and misaligned operands; rows without an expert, which hold NaN
throughout. Bounds as for the dense products (ff_util)."""
import pytest
import torch

from ff_util import ACTS, TYPES, acc_error, act64, assert_within, matrix, rounding, slope64

pytestmark = pytest.mark.gpu

# rows of each expert: none, one, around the 16- and 64-row steps and the 128- and 256-row tiles
COUNTS = [[1], [0, 3, 0], [5, 0, 17], [64, 128, 256, 16], [63, 65, 127, 129, 1, 15], [255, 0, 257, 33],
          [300, 513, 31, 96], [1000, 2, 700], [2] * 40, [0] * 70 + [9]]
# (N, K)
EXTENTS = [(1, 1), (64, 64), (200, 136), (256, 256), (130, 1000), (1025, 127), (520, 72), (8, 2048)]


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


def offsets_of(counts, first=0):
    o = torch.tensor([first] + counts).cumsum(0)
    return o.to(torch.int32).cuda(), o.tolist()


def weights(experts, K, N, t, seed, layout="col", pad=0, offset=0, gap=0):
    """experts x K x N, each with `pad` NaN after every line and `gap` NaN after each expert."""
    lines, length = (N, K) if layout == "col" else (K, N)
    one = lines * (length + pad) + gap
    store = torch.full((offset + experts * one,), float("nan"), dtype=t, device="cuda")
    view = store[offset:].as_strided((experts, lines, length), (one, length + pad, 1))
    gen = torch.Generator("cuda").manual_seed(seed)
    view.copy_((torch.randn(experts, lines, length, generator=gen, device="cuda") * K ** -0.5).to(t))
    return view.transpose(1, 2) if layout == "col" else view


def rows_with_gaps(rows, cols, t, seed, bounds, pad=0, offset=0, scale=1.0):
    """Normal rows, NaN before the first expert's and after the last one's."""
    x = matrix(rows, cols, t, seed, pad=pad, offset=offset, scale=scale)
    x[:bounds[0]] = float("nan")
    x[bounds[-1]:] = float("nan")
    return x


def sentinel(rows, cols, t, pad=0, offset=0):
    return matrix(rows, cols, t, 99, pad=pad, offset=offset).fill_(7.0)


def accumulation(t, K):
    """Relative bound on a K-long sum: as the dense kernels' in the tensor cores; for fp32 chains of
    128 fused multiply-adds, each added to a running total, so that no addend takes more than
    min(K, 128) + ceil(K / 128) roundings of half a step."""
    if t != torch.float32:
        return acc_error(t, K)
    return (min(K, 128) + -(-K // 128)) * 2.0 ** -24


def untouched(y, bounds):
    assert (y[:bounds[0]] == 7).all() and (y[bounds[-1]:] == 7).all()


def check_product(h, x, w, offsets, bounds, out):
    t, K = x.dtype, x.shape[1]
    y = h.expert_matmul(x, w, offsets, out=out)
    assert y is out
    for e in range(w.shape[0]):
        a, b = bounds[e], bounds[e + 1]
        xd, wd = x[a:b].double(), w[e].double()
        want = xd @ wd
        D = xd.abs() @ wd.abs()
        assert_within(y[a:b], want, 1.01 * accumulation(t, K) * D + rounding(want, t), "y of %d" % e)
    untouched(y, bounds)


def check_backward(h, dy, x, w, offsets, bounds, out, need=(True, True)):
    t, N = x.dtype, w.shape[2]
    dx, dw = h.expert_matmul_backward(dy, x, w, offsets, need=need, out=out)
    for e in range(w.shape[0]):
        a, b = bounds[e], bounds[e + 1]
        xd, wd, d = x[a:b].double(), w[e].double(), dy[a:b].double()
        if need[0]:
            want = d @ wd.t()
            bound = accumulation(t, N) * (d.abs() @ wd.abs().t())
            assert_within(dx[a:b], want, bound * 1.01 + rounding(want, t), "dx of %d" % e)
        if need[1]:
            want = xd.t() @ d
            bound = accumulation(t, b - a) * (xd.abs().t() @ d.abs())
            assert_within(dw[e], want, bound * 1.01 + rounding(want, t), "dw of %d" % e)
    if need[0]:
        untouched(dx, bounds)
    else:
        assert dx is None
    assert need[1] or dw is None
    return dx, dw


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("N,K", EXTENTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_product(h, counts, N, K, dtype):
    t = TYPES[dtype]
    offsets, bounds = offsets_of(counts, 2)
    rows = bounds[-1] + 3
    x = rows_with_gaps(rows, K, t, 1, bounds)
    w = weights(len(counts), K, N, t, 2)
    check_product(h, x, w, offsets, bounds, sentinel(rows, N, t))
    dy = rows_with_gaps(rows, N, t, 3, bounds)
    check_backward(h, dy, x, w, offsets, bounds, sentinel(rows, K, t))


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("pad,offset,gap", [(0, 0, 0), (8, 8, 16), (3, 1, 0), (8, 0, 5), (4, 4, 4), (2, 0, 0)])
@pytest.mark.parametrize("counts", [[5, 0, 300, 64], [40]], ids=str)
@pytest.mark.parametrize("N,K", [(200, 136), (264, 72), (133, 65), (132, 68), (4, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_product_layouts(h, counts, N, K, layout, pad, offset, gap, dtype):
    t = TYPES[dtype]
    offsets, bounds = offsets_of(counts, 1)
    rows = bounds[-1] + 2
    x = rows_with_gaps(rows, K, t, 1, bounds, pad, offset)
    w = weights(len(counts), K, N, t, 2, layout, pad, offset, gap)
    check_product(h, x, w, offsets, bounds, sentinel(rows, N, t, pad, offset))
    dy = rows_with_gaps(rows, N, t, 3, bounds, pad, offset)
    dx, dw = check_backward(h, dy, x, w, offsets, bounds, sentinel(rows, K, t, pad, offset))
    assert (dw.stride(1) == 1) == (layout == "col") or min(N, K) == 1


@pytest.mark.parametrize("layout", ["row", "col"])
def test_long_f32_sums(h, layout):
    """Addends of one sign, whose roundings grow with the running total."""
    t = torch.float32
    offsets, bounds = offsets_of([5000, 3, 2000])
    x = matrix(bounds[-1], 3001, t, 1).abs_()
    w = weights(3, 3001, 70, t, 2, layout).abs_()
    check_product(h, x, w, offsets, bounds, sentinel(bounds[-1], 70, t))
    dy = matrix(bounds[-1], 70, t, 3).abs_()
    check_backward(h, dy, x, w, offsets, bounds, sentinel(bounds[-1], 3001, t))


def test_parts(h):
    offsets, bounds = offsets_of([5, 70])
    x, w = matrix(75, 72, torch.bfloat16, 1), weights(2, 72, 40, torch.bfloat16, 2)
    dy = matrix(75, 40, torch.bfloat16, 3)
    for need in ((True, False), (False, True), (False, False)):
        check_backward(h, dy, x, w, offsets, bounds, sentinel(75, 72, torch.bfloat16), need)


def check_gated(h, x, wg, wu, offsets, bounds, act, save=True):
    t, K, F = x.dtype, x.shape[1], wg.shape[2]
    out = sentinel(x.shape[0], F, t)
    got = h.expert_gated(x, wg, wu, offsets, activation=act, out=out, save=save)
    y, gate, up = got if save else (got, None, None)
    for e in range(wg.shape[0]):
        a, b = bounds[e], bounds[e + 1]
        xd = x[a:b].double()
        gd, ud = xd @ wg[e].double(), xd @ wu[e].double()
        err = accumulation(t, K)
        eg, eu = err * (xd.abs() @ wg[e].double().abs()), err * (xd.abs() @ wu[e].double().abs())
        if save:
            assert_within(gate[a:b], gd, eg + rounding(gd, t) * 1.01, "gate of %d" % e)
            assert_within(up[a:b], ud, eu + rounding(ud, t) * 1.01, "up of %d" % e)
        f = act64(gd, act)
        ef = 1.2 * eg + 2.0 ** -20 * (gd.abs() + 1)
        want = f * ud
        bound = ef * (ud.abs() + eu) + f.abs() * eu + 2.0 ** -23 * want.abs()
        assert_within(y[a:b], want, bound * 1.01 + rounding(want, t), "h of %d" % e)
    untouched(y, bounds)
    return y


def check_gated_backward(h, dh, x, wg, wu, gate, up, offsets, bounds, act, need=(True, True, True)):
    t, F = x.dtype, wg.shape[2]
    out = sentinel(x.shape[0], x.shape[1], t)
    dx, dwg, dwu = h.expert_gated_backward(dh, x, wg, wu, gate, up, offsets, activation=act, need=need,
                                           out=out)
    for e in range(wg.shape[0]):
        a, b = bounds[e], bounds[e + 1]
        xd, g, u, d = (v[a:b].double() for v in (x, gate, up, dh))
        f, s = act64(g, act), slope64(g, act)
        dg, du = d * u * s, d * f
        # slopes in fp32, and rounded as operands of their type
        eg = 2.0 ** -19 * (1 + g.abs()) * (d * u).abs() + rounding(dg, t) * 1.01
        eu = 2.0 ** -19 * (1 + g.abs()) * d.abs() + rounding(du, t) * 1.01
        if need[0]:
            wgd, wud = wg[e].double().t(), wu[e].double().t()
            want = dg @ wgd + du @ wud
            D = (dg.abs() + eg) @ wgd.abs() + (du.abs() + eu) @ wud.abs()
            bound = eg @ wgd.abs() + eu @ wud.abs() + accumulation(t, 2 * F) * D
            assert_within(dx[a:b], want, bound * 1.01 + rounding(want, t), "dx of %d" % e)
        for dw, v, ev, needed, what in ((dwg, dg, eg, need[1], "dwg"), (dwu, du, eu, need[2], "dwu")):
            if not needed:
                assert dw is None
                continue
            want = xd.t() @ v
            bound = xd.abs().t() @ ev + accumulation(t, b - a) * (xd.abs().t() @ (v.abs() + ev))
            assert_within(dw[e], want, bound * 1.01 + rounding(want, t), "%s of %d" % (what, e))
    if need[0]:
        untouched(dx, bounds)


@pytest.mark.parametrize("counts", COUNTS, ids=str)
@pytest.mark.parametrize("F,K", [(1, 1), (64, 64), (200, 136), (130, 1000), (1025, 127), (520, 72)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_gated(h, counts, F, K, dtype):
    t = TYPES[dtype]
    offsets, bounds = offsets_of(counts, 2)
    rows = bounds[-1] + 3
    x = rows_with_gaps(rows, K, t, 1, bounds)
    wg, wu = weights(len(counts), K, F, t, 2), weights(len(counts), K, F, t, 3)
    check_gated(h, x, wg, wu, offsets, bounds, "silu", save=(F + K) % 2 == 0)
    dh, gate, up = (rows_with_gaps(rows, F, t, s, bounds) for s in (4, 5, 6))
    check_gated_backward(h, dh, x, wg, wu, gate, up, offsets, bounds, "silu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_activations(h, act, dtype):
    t = TYPES[dtype]
    offsets, bounds = offsets_of([33, 0, 150])
    x = matrix(183, 136, t, 1, scale=3.0)
    wg, wu = (weights(3, 136, 200, t, s) for s in (2, 3))
    check_gated(h, x, wg, wu, offsets, bounds, act)
    dh, gate, up = (matrix(183, 200, t, s) for s in (4, 5, 6))
    gate[0, :8] = 0
    check_gated_backward(h, dh, x, wg, wu, gate, up, offsets, bounds, act)


@pytest.mark.parametrize("layout", ["row", "col"])
@pytest.mark.parametrize("pad,offset,gap", [(0, 0, 0), (8, 8, 16), (3, 1, 0), (4, 4, 4), (2, 2, 0)])
@pytest.mark.parametrize("F,K", [(200, 136), (133, 65), (144, 64), (132, 68)])
@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_gated_layouts(h, F, K, layout, pad, offset, gap, dtype):
    t = TYPES[dtype]
    offsets, bounds = offsets_of([5, 0, 200, 64], 1)
    rows = bounds[-1] + 2
    x = rows_with_gaps(rows, K, t, 1, bounds, pad, offset)
    wg, wu = (weights(4, K, F, t, s, layout, pad, offset, gap) for s in (2, 3))
    check_gated(h, x, wg, wu, offsets, bounds, "gelu")
    both = rows_with_gaps(rows, 2 * F, t, 5, bounds, pad, offset)
    dh = rows_with_gaps(rows, F, t, 4, bounds, pad, offset)
    check_gated_backward(h, dh, x, wg, wu, both[:, :F], both[:, F:], offsets, bounds, "gelu_tanh")


def test_gated_one_weight_buffer(h):
    """Both weights as parts of one tensor, expert by expert."""
    offsets, bounds = offsets_of([5, 90])
    x = matrix(95, 128, torch.bfloat16, 1)
    w = weights(2, 128, 400, torch.bfloat16, 2)
    check_gated(h, x, w[:, :, :200], w[:, :, 200:], offsets, bounds, "silu")
    w = weights(2, 128, 400, torch.bfloat16, 2, "row")
    check_gated(h, x, w[:, :, :200], w[:, :, 200:], offsets, bounds, "silu")


def test_gated_parts(h):
    offsets, bounds = offsets_of([5, 70])
    x = matrix(75, 72, torch.bfloat16, 1)
    wg, wu = (weights(2, 72, 40, torch.bfloat16, s) for s in (2, 3))
    dh, gate, up = (matrix(75, 40, torch.bfloat16, s) for s in (4, 5, 6))
    for need in ((True, False, False), (False, True, False), (False, False, True), (False,) * 3):
        check_gated_backward(h, dh, x, wg, wu, gate, up, offsets, bounds, "silu", need)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_stay_with_their_expert(h, dtype):
    """NaN and infinities in one expert's rows or weights reach that expert's results alone."""
    t = TYPES[dtype]
    counts = [33, 47, 21]
    offsets, bounds = offsets_of(counts)
    x, dy = matrix(101, 72, t, 1), matrix(101, 136, t, 2)
    w = weights(3, 72, 136, t, 3)
    clean = h.expert_matmul(x, w, offsets), *h.expert_matmul_backward(dy, x, w, offsets)
    x[bounds[1]:bounds[2]] = float("inf")
    dy[bounds[1]:bounds[2]] = float("nan")
    w[1] = float("-inf")
    dirty = h.expert_matmul(x, w, offsets), *h.expert_matmul_backward(dy, x, w, offsets)
    for i in range(2):
        for e in (0, 2):
            a, b = bounds[e], bounds[e + 1]
            assert torch.equal(clean[i][a:b], dirty[i][a:b])
        assert not torch.isfinite(dirty[i][bounds[1]:bounds[2]]).any()
    assert torch.equal(clean[2][0], dirty[2][0]) and torch.equal(clean[2][2], dirty[2][2])
    assert torch.isnan(dirty[2][1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_offsets_stay_inside(h, dtype):
    """Offsets outside the rows are taken as clamped, and an expert that would end before its start
    has no rows; nothing outside the matrices is written."""
    t = TYPES[dtype]
    store = torch.full((120, 72), 7.0, dtype=t, device="cuda")
    out = store[10:110]
    x, w = matrix(100, 64, t, 1), weights(4, 64, 72, t, 2)
    want = [x.float() @ w[e].float() for e in range(4)]
    for o, bounds in (([-5, 20, 60, 90, 1000], [0, 20, 60, 90, 100]),
                      ([0, 50, 50, 2 ** 31 - 1, -2 ** 31], [0, 50, 50, 100, 100]),
                      ([0, 60, 40, 80, 100], [0, 60, 60, 80, 100])):
        out.fill_(7.0)
        h.expert_matmul(x, w, torch.tensor(o, dtype=torch.int32, device="cuda"), out=out)
        for e in range(4):
            a, b = bounds[e], bounds[e + 1]
            assert torch.allclose(out[a:b].float(), want[e][a:b], atol=0.05, rtol=0.02)
        assert (store[:10] == 7).all() and (store[110:] == 7).all()
        dy = matrix(100, 72, t, 3)
        dx, dw = h.expert_matmul_backward(dy, x, w, torch.tensor(o, dtype=torch.int32, device="cuda"))
        assert torch.isfinite(dw).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_empty(h, dtype):
    t = TYPES[dtype]
    e = lambda *s: torch.empty(*s, dtype=t, device="cuda")
    offsets, _ = offsets_of([0, 0])
    w = weights(2, 24, 40, t, 1)
    assert h.expert_matmul(e(0, 24), w, offsets).shape == (0, 40)
    dx, dw = h.expert_matmul_backward(e(0, 40), e(0, 24), w, offsets)
    assert dx.shape == (0, 24) and (dw == 0).all()
    dx, dwg, dwu = h.expert_gated_backward(e(0, 40), e(0, 24), w, w, e(0, 40), e(0, 40), offsets)
    assert dx.shape == (0, 24) and (dwg == 0).all() and (dwu == 0).all()
    dx, dw = h.expert_matmul_backward(matrix(5, 40, t, 1), matrix(5, 24, t, 2), w, offsets,
                                      out=sentinel(5, 24, t))
    assert (dx == 7).all() and (dw == 0).all()  # rows, but no expert's
    offsets, bounds = offsets_of([2, 0], 1)
    y = h.expert_matmul(e(5, 0), e(2, 0, 40), offsets, out=sentinel(5, 40, t))
    assert (y[1:3] == 0).all() and (y[0] == 7).all() and (y[3:] == 7).all()
    dx, dw = h.expert_matmul_backward(e(5, 0), matrix(5, 24, t, 1), e(2, 24, 0), offsets,
                                      out=sentinel(5, 24, t))
    assert (dx[1:3] == 0).all() and (dx[3:] == 7).all() and dw.shape == (2, 24, 0)
    y, gate, up = h.expert_gated(e(5, 0), e(2, 0, 40), e(2, 0, 40), offsets, activation="sigmoid", save=True)
    assert (y[1:3] == 0).all() and (gate[1:3] == 0).all() and (up[1:3] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_experts(h, dtype):
    """1024 experts, most without rows."""
    t = TYPES[dtype]
    counts = [0] * 1024
    for e in (0, 3, 500, 1023):
        counts[e] = e % 37 + 1
    offsets, bounds = offsets_of(counts)
    x, w = matrix(bounds[-1], 72, t, 1), weights(1024, 72, 80, t, 2)
    y = h.expert_matmul(x, w, offsets)
    dy = matrix(bounds[-1], 80, t, 3)
    dx, dw = h.expert_matmul_backward(dy, x, w, offsets)
    for e in range(1024):
        a, b = bounds[e], bounds[e + 1]
        if a == b:
            assert (dw[e] == 0).all()
            continue
        xd, wd, d = x[a:b].double(), w[e].double(), dy[a:b].double()
        for got, want, D, K in ((y[a:b], xd @ wd, xd.abs() @ wd.abs(), 72),
                                (dx[a:b], d @ wd.t(), d.abs() @ wd.abs().t(), 80),
                                (dw[e], xd.t() @ d, xd.abs().t() @ d.abs(), b - a)):
            assert_within(got, want, 1.01 * acc_error(t, K) * D + rounding(want, t))


def test_gradients_against_differences(h):
    """The gated pair's gradients along random directions against central differences of the
    definition in 64 bits, in f16. Each gradient's element is off by the roundings of gate, up, slope
    and itself, 2^-11 each (gate's and up's with factors up to 3): at random, so at most 5 deviations
    of 2^-11 (3 + 3 + 1 + 1) times the gradient's norm, 2e-2."""
    t = torch.float16
    offsets, bounds = offsets_of([40, 0, 23])
    x = matrix(63, 64, t, 1)
    wg, wu = (weights(3, 64, 96, t, s) for s in (2, 3))
    dh = matrix(63, 96, t, 4)

    def loss(a, b, c):
        out = 0.0
        for e in range(3):
            r = slice(bounds[e], bounds[e + 1])
            gd, ud = a[r] @ b[e], a[r] @ c[e]
            out = out + (act64(gd, "silu") * ud * dh[r].double()).sum()
        return float(out)

    _, gate, up = h.expert_gated(x, wg, wu, offsets, activation="silu", save=True)
    grads = h.expert_gated_backward(dh, x, wg, wu, gate, up, offsets, activation="silu")
    args = [v.double() for v in (x, wg, wu)]
    for i in range(3):
        d = torch.randn(args[i].shape, generator=torch.Generator("cuda").manual_seed(i), device="cuda",
                        dtype=torch.float64)
        step = 2.0 ** -10
        up_, down = list(args), list(args)
        up_[i], down[i] = args[i] + step * d, args[i] - step * d
        slope = (loss(*up_) - loss(*down)) / (2 * step)
        got = float((grads[i].double() * d).sum())
        size = float((grads[i].double() ** 2).sum().sqrt())
        assert abs(got - slope) <= 2e-2 * size


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_captured_with_other_offsets(h, dtype):
    """One captured call serves every distribution of the rows; two graphs share the handle's
    buffers, which a larger call outgrows."""
    t = TYPES[dtype]
    x, dy = matrix(300, 133, t, 1), matrix(300, 72, t, 2)  # (rows TMA cannot address: copied first)
    w = weights(4, 133, 72, t, 3)
    offsets = torch.zeros(5, dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(stream):
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                outs = h.expert_matmul(x, w, offsets), *h.expert_matmul_backward(dy, x, w, offsets)
            graphs.append((graph, outs))
    torch.cuda.synchronize()
    big = matrix(5000, 133, t, 4)
    h.expert_matmul(big, w, offsets_of([5000, 0, 0, 0])[0])
    for counts in ([100, 0, 150, 50], [0, 300, 0, 0], [1, 1, 1, 200]):
        o, bounds = offsets_of(counts)
        offsets.copy_(o)
        for graph, outs in graphs:
            graph.replay()
            torch.cuda.synchronize()
            eager = h.expert_matmul(x, w, o), *h.expert_matmul_backward(dy, x, w, o)
            live = bounds[-1]
            assert torch.equal(outs[0][:live], eager[0][:live])
            assert torch.equal(outs[1][:live], eager[1][:live])
            assert torch.equal(outs[2], eager[2])
    assert h.status() == 0


def test_on_another_stream(h):
    offsets, bounds = offsets_of([40, 60])
    x, w = matrix(100, 128, torch.bfloat16, 1), weights(2, 128, 136, torch.bfloat16, 2)
    want = h.expert_matmul(x, w, offsets), h.expert_gated(x, w, w, offsets)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    got = h.expert_matmul(x, w, offsets, stream=stream), h.expert_gated(x, w, w, offsets, stream=stream)
    torch.cuda.current_stream().wait_stream(stream)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("stall", [1, 2, 3, 6, 7])
@pytest.mark.parametrize("counts", [[400, 33], [70, 5, 330]], ids=str)
def test_bounded_waits_expire_and_the_next_call_is_right(g, counts, stall):
    """A loader that issues nothing, or stops with copies in flight -- ragged blocks' among them --
    ends in a status, and the handle works on."""
    t = torch.bfloat16
    hh = g.Gemm(0)
    hh.set_option("wait_timeout_us", 20000)
    offsets, bounds = offsets_of(counts)
    rows = bounds[-1]
    x, w, dy = matrix(rows, 512, t, 1), weights(len(counts), 512, 256, t, 2), matrix(rows, 256, t, 3)

    def done(f):
        r = f()
        torch.cuda.synchronize()
        return r

    calls = {"product": lambda: done(lambda: hh.expert_matmul(x, w, offsets)),
             "gated": lambda: done(lambda: hh.expert_gated(x, w, w, offsets)),
             "dw": lambda: done(lambda: hh.expert_matmul_backward(dy, x, w, offsets, need=(False, True)))}

    for name, call in calls.items():
        right = call()
        assert hh.status() == 0
        hh.set_option("fault_stall_producer", stall)
        call()
        assert hh.status() == 6, name
        hh.set_option("fault_stall_producer", 0)
        again = call()
        assert hh.status() == 0
        a, b = (right, again) if torch.is_tensor(right) else (right[1], again[1])
        assert torch.equal(a, b), name
    hh.close()


def test_refusals(g, h):
    t = torch.bfloat16
    x, w = torch.zeros(6, 16, dtype=t, device="cuda"), torch.zeros(2, 16, 24, dtype=t, device="cuda")
    offsets = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    dy = torch.zeros(6, 24, dtype=t, device="cuda")
    with pytest.raises(TypeError):
        h.expert_matmul(x.half(), w, offsets)
    with pytest.raises(TypeError):
        h.expert_matmul(x, w, offsets.long())
    with pytest.raises(ValueError):
        h.expert_matmul(x, w, offsets[:2])
    with pytest.raises(ValueError):
        h.expert_matmul(x, w[0], offsets)
    with pytest.raises(ValueError):
        h.expert_matmul(x[:, :8], w, offsets)
    with pytest.raises(ValueError):
        h.expert_matmul(x, w, offsets.cpu())
    with pytest.raises(ValueError):
        h.expert_matmul(x, w[:, ::2, ::2], offsets)
    with pytest.raises(TypeError):
        h.expert_matmul(x, w, offsets, out=dy.float())
    with pytest.raises(ValueError):
        h.expert_matmul(x, w, offsets, out=dy[:5])
    with pytest.raises(g.GemmError, match="INVALID_ARG"):  # one set of weights for all experts
        h.expert_matmul(x, w[:1].expand(2, 16, 24), offsets)
    with pytest.raises(g.GemmError, match="INVALID_ARG"):
        square = torch.zeros(2, 16, 16, dtype=t, device="cuda")
        h.expert_matmul(x, square, offsets, out=x)
    with pytest.raises(ValueError):
        h.expert_gated(x, w, w[:, :, :16], offsets)
    with pytest.raises(ValueError):
        h.expert_gated(x, w, torch.zeros(2, 24, 16, dtype=t, device="cuda").transpose(1, 2), offsets)
    with pytest.raises(ValueError):
        h.expert_gated(x, w, w, offsets, activation="swish")
    with pytest.raises(TypeError):
        h.expert_gated_backward(dy.float(), x, w, w, dy, dy, offsets)
    with pytest.raises(ValueError):
        h.expert_matmul_backward(dy[:, :8], x, w, offsets)
    many = torch.zeros(1025, 8, 8, dtype=t, device="cuda")
    with pytest.raises(g.GemmError, match="UNSUPPORTED"):
        h.expert_matmul(x[:, :8], many, torch.zeros(1026, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("counts", [[0, 3, 0, 0, 1, 0], [0] * 5 + [40], [7] + [0] * 200], ids=str)
def test_copied_weights_of_few_experts(h, counts):
    """Rows that TMA cannot address: only the weights of experts that have rows are copied, call by
    call, and others' may hold anything."""
    t = torch.bfloat16
    w = weights(len(counts), 1001, 75, t, 2)
    for e, n in enumerate(counts):
        if n == 0:
            w[e] = float("nan")
    for turn in (counts, counts[::-1]):
        offsets, bounds = offsets_of(turn)
        x, dy = matrix(bounds[-1], 1001, t, 1), matrix(bounds[-1], 75, t, 3)
        here = w if turn is counts else w.flip(0)
        check_product(h, x, here, offsets, bounds, sentinel(bounds[-1], 75, t))
        check_backward(h, dy, x, here, offsets, bounds, sentinel(bounds[-1], 1001, t))
        check_gated(h, x, here, here.clone(), offsets, bounds, "silu")
