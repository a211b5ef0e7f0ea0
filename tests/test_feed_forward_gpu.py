"""The feed-forward operators on the GPU against their definitions in 64 bits: a product with
bias, activation and residual, the gated pair of projections, and their backward passes. Sizes
around every tile edge, empty extents, both layouts, padded and misaligned operands, each
type; gradients against the formulas and against differences of the forward pass."""
import pytest
import torch

from ff_util import (ACTS, TYPES, UNIT, acc_error, act64, assert_within, matrix, rounding,
                     slope64)

pytestmark = pytest.mark.gpu

# (M, N, K): one row to several tiles, odd and ragged extents, K around the 64-long K-blocks
SIZES = [(1, 1, 1), (1, 64, 64), (1, 4096, 512), (2, 17, 33), (3, 130, 1000), (7, 1025, 127),
         (16, 128, 64), (17, 256, 200), (33, 300, 1024), (64, 512, 136), (65, 127, 72),
         (100, 1024, 2048), (127, 129, 129), (128, 256, 1), (129, 1000, 65), (200, 8, 4096),
         (255, 257, 64), (256, 2048, 256), (257, 96, 1023), (513, 640, 320), (1023, 1025, 17),
         (1030, 520, 96)]
SMALL = [(1, 1, 1), (3, 130, 100), (17, 256, 200), (65, 127, 72), (257, 96, 129), (300, 520, 96)]


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    hh = g.Gemm(0)
    yield hh
    assert hh.status() == 0
    hh.close()


def operands(M, N, K, dtype, seed, a_layout="row", b_layout="col", pad=0, offset=0):
    t = TYPES[dtype]
    a = matrix(M, K, t, seed, a_layout, pad, offset)
    b = matrix(K, N, t, seed + 1, b_layout, pad, offset, scale=max(K, 1) ** -0.5)
    return a, b


def check_epilogue(h, a, b, act, bias, residual, out_dtype=None, precision="default", save=True,
                   out=None):
    M, K = a.shape
    N = b.shape[1]
    r64 = None if residual is None else residual.double()  # (residual may be the output)
    got = h.matmul_epilogue(a, b, bias=bias, activation=act, residual=residual, out=out,
                            out_dtype=out_dtype, precision=precision, save=save)
    torch.cuda.synchronize()
    y, pre = got if save else (got, None)
    z = a.double() @ b.double()
    e = acc_error(a.dtype, K, precision) * (a.double().abs() @ b.double().abs())
    if bias is not None:
        z = z + bias.double()
        e = e + 2.0 ** -23 * (z.abs() + bias.double().abs())
    if save:
        assert_within(pre, z, e + rounding(z, pre.dtype), "pre")
    want = act64(z, act)
    e = 1.2 * e + 2.0 ** -20 * (z.abs() + 1)
    if residual is not None:
        want = want + r64
        e = e + 2.0 ** -23 * (want.abs() + r64.abs())
    assert_within(y, want, e * 1.01 + rounding(want, y.dtype), "y")
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_epilogue_sizes(h, M, N, K, dtype):
    a, b = operands(M, N, K, dtype, 10 * M + N)
    bias = matrix(1, N, TYPES[dtype], 5)[0]
    residual = matrix(M, N, TYPES[dtype], 6)
    check_epilogue(h, a, b, "silu", bias, residual)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", [(5, 200, 136), (150, 264, 136), (300, 520, 200)])
def test_epilogue_activations(h, M, N, K, dtype, act):
    a, b = operands(M, N, K, dtype, 77)
    a = a * 3  # well into the activations' tails
    check_epilogue(h, a, b, act, matrix(1, N, torch.float32, 5)[0], None)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("b_layout", ["row", "col"])
@pytest.mark.parametrize("a_layout", ["row", "col"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (3, 1)])
@pytest.mark.parametrize("M,N,K", [(9, 136, 72), (260, 200, 136)])
def test_epilogue_layouts(h, M, N, K, a_layout, b_layout, pad, offset, dtype):
    t = TYPES[dtype]
    a, b = operands(M, N, K, dtype, 31, a_layout, b_layout, pad, offset)
    bias = matrix(1, N + 1, t, 5)[0][1:]  # aligned to its element only
    residual = matrix(M, N, t, 6, pad=pad, offset=offset)
    store = torch.full((M, N + 5), 7.0, dtype=t, device="cuda")
    check_epilogue(h, a, b, "gelu", bias, residual, out=store[:, :N])
    assert (store[:, N:] == 7).all()  # nothing written past the rows


@pytest.mark.parametrize("pieces", range(16))
def test_epilogue_parts(h, pieces):
    """Every combination of bias, activation, residual and kept pre-activation."""
    for M in (4, 300):
        a, b = operands(M, 264, 128, "bf16", 3)
        bias = matrix(1, 264, torch.bfloat16, 5)[0] if pieces & 1 else None
        residual = matrix(M, 264, torch.bfloat16, 6) if pieces & 2 else None
        check_epilogue(h, a, b, "relu" if pieces & 4 else None, bias, residual,
                       save=bool(pieces & 8))


@pytest.mark.parametrize("in_dtype,out_dtype", [("bf16", "f32"), ("f16", "f32"), ("bf16", "f16"),
                                                ("f16", "bf16"), ("f32", "bf16"), ("f32", "f16")])
@pytest.mark.parametrize("M", [3, 270])
def test_epilogue_output_types(h, M, in_dtype, out_dtype):
    a, b = operands(M, 200, 96, in_dtype, 8)
    for bias_dtype in ("f32", "f16", "bf16"):
        check_epilogue(h, a, b, "gelu_tanh", matrix(1, 200, TYPES[bias_dtype], 5)[0],
                       matrix(M, 200, TYPES[out_dtype], 6), out_dtype=out_dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(1, 64), (6, 70), (300, 264), (300, 261)])
def test_epilogue_residual_in_place(h, M, N, dtype):
    a, b = operands(M, N, 128, dtype, 8)
    r = matrix(M, N, TYPES[dtype], 6)
    y = check_epilogue(h, a, b, None, None, r, out=r, save=False)
    assert y.data_ptr() == r.data_ptr()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [5, 300])
def test_epilogue_empty_extents(h, M, dtype):
    t = TYPES[dtype]
    bias = matrix(1, 40, t, 5)[0]
    # K == 0: the epilogue of an empty sum
    a, b = torch.empty(M, 0, dtype=t, device="cuda"), torch.empty(0, 40, dtype=t, device="cuda")
    y, pre = h.matmul_epilogue(a, b, bias=bias, activation="gelu_tanh", save=True)
    assert torch.equal(pre, bias.expand(M, 40))
    want = act64(bias.double(), "gelu_tanh").expand(M, 40)
    assert_within(y, want, rounding(want, t) + 2.0 ** -20, "y")
    # no rows, no columns
    z = torch.empty(0, 64, dtype=t, device="cuda")
    assert h.matmul_epilogue(z, matrix(64, 40, t, 1), bias=bias, activation="silu").shape == (0, 40)
    assert h.matmul_epilogue(matrix(M, 64, t, 1), torch.empty(64, 0, dtype=t, device="cuda"),
                             activation="silu").shape == (M, 0)


def test_epilogue_tf32(h):
    for M in (4, 300):
        a, b = operands(M, 130, 200, "f32", 8)
        check_epilogue(h, a, b, "silu", matrix(1, 130, torch.float32, 5)[0], None, precision="tf32")


def test_epilogue_special_values(h):
    """NaN and infinities follow the formula; a NaN stays in its own row."""
    for M in (4, 300):
        a, b = operands(M, 136, 64, "bf16", 8)
        a[1, 3] = float("nan")
        a[2, :] = 0
        bias = torch.zeros(136, device="cuda")
        bias[5] = float("inf")
        y = h.matmul_epilogue(a, b, bias=bias, activation="silu").float()
        assert torch.isnan(y[1]).all()
        assert torch.isinf(y[0, 5]) and torch.isfinite(y[0, :5]).all()
        assert (y[2, :5] == 0).all() and torch.isinf(y[2, 5])
        r = h.matmul_epilogue(a, b, activation="relu").float()
        assert torch.isnan(r[1]).all() and not torch.isnan(r[0]).any()


# -------------------------------------------------------------------------- gated

def check_gated(h, x, wg, wu, act, save, precision="default"):
    K = x.shape[1]
    got = h.gated(x, wg, wu, activation=act, save=save, precision=precision)
    torch.cuda.synchronize()
    out = got[0] if save else got
    xd = x.double()
    g, u = xd @ wg.double(), xd @ wu.double()
    e = acc_error(x.dtype, K, precision)
    eg, eu = e * (xd.abs() @ wg.double().abs()), e * (xd.abs() @ wu.double().abs())
    if save:
        assert_within(got[1], g, eg + rounding(g, x.dtype), "gate")
        assert_within(got[2], u, eu + rounding(u, x.dtype), "up")
    f = act64(g, act)
    ef = 1.2 * eg + 2.0 ** -20 * (g.abs() + 1)
    want = f * u
    bound = ef * (u.abs() + eu) + f.abs() * eu + 2.0 ** -23 * want.abs()
    assert_within(out, want, bound * 1.01 + rounding(want, x.dtype), "h")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,F,K", SIZES)
def test_gated_sizes(h, M, F, K, dtype):
    x, wg = operands(M, F, K, dtype, 10 * M + F)
    wu = matrix(K, F, TYPES[dtype], 9, "col", scale=max(K, 1) ** -0.5)
    check_gated(h, x, wg, wu, "silu", save=(M + F) % 2 == 0)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M,F,K", [(5, 200, 136), (300, 264, 136)])
def test_gated_activations(h, M, F, K, act):
    x, wg = operands(M, F, K, "bf16", 77)
    wu = matrix(K, F, torch.bfloat16, 9, "col", scale=K ** -0.5)
    check_gated(h, x * 3, wg, wu, act, save=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("w_layout", ["row", "col"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (3, 1)])
@pytest.mark.parametrize("M,F,K", [(9, 136, 72), (260, 200, 136)])
def test_gated_layouts(h, M, F, K, w_layout, pad, offset, dtype):
    x, wg = operands(M, F, K, dtype, 31, "row", w_layout, pad, offset)
    wu = matrix(K, F, TYPES[dtype], 9, w_layout, pad + 8, offset, scale=K ** -0.5)
    check_gated(h, x, wg, wu, "gelu", save=True)


@pytest.mark.parametrize("M", [1, 300])
def test_gated_one_weight_buffer(h, M):
    """Both weights as halves of one tensor, by rows and by columns."""
    x = matrix(M, 128, torch.bfloat16, 1)
    w = matrix(400, 128, torch.bfloat16, 2, scale=0.1)
    check_gated(h, x, w[:200].t(), w[200:].t(), "silu", save=True)
    w = matrix(128, 400, torch.bfloat16, 2, scale=0.1)
    check_gated(h, x, w[:, :200], w[:, 200:], "silu", save=True)


def test_gated_empty_extents(h):
    t = torch.bfloat16
    e = lambda *s: torch.empty(*s, dtype=t, device="cuda")
    out, g, u = h.gated(e(3, 0), e(0, 40), e(0, 40), activation="sigmoid", save=True)
    assert (out == 0).all() and (g == 0).all() and (u == 0).all()
    assert h.gated(e(0, 64), e(64, 40), e(64, 40)).shape == (0, 40)
    assert h.gated(e(3, 64), e(64, 0), e(64, 0)).shape == (3, 0)


# ----------------------------------------------------------------------- backward

def check_epilogue_backward(h, dy, a, b, pre, act, need=(True, True, True), bias_dtype=None):
    M, K = a.shape
    N = b.shape[1]
    da, db, dbias = h.matmul_epilogue_backward(dy, a, b, pre=pre, activation=act, need=need,
                                               bias_dtype=bias_dtype)
    torch.cuda.synchronize()
    dz = dy.double()
    ez = 0 * dz
    if act not in (None, "none"):
        dz = dz * slope64(pre.double(), act)
        ez = 2.0 ** -19 * (1 + pre.double().abs()) * dy.double().abs()
    if dbias is not None:
        want = dz.sum(0)
        bound = (M + 16) * 2.0 ** -24 * dz.abs().sum(0) + ez.sum(0)
        assert_within(dbias, want, bound + rounding(want, dbias.dtype), "dbias")
    ez = ez + rounding(dz, a.dtype)  # dz as an operand of its type
    ad, bd = a.double(), b.double()
    if da is not None:
        want = dz @ bd.t()
        bound = ez @ bd.abs().t() + acc_error(a.dtype, N) * ((dz.abs() + ez) @ bd.abs().t())
        assert_within(da, want, bound * 1.01 + rounding(want, a.dtype), "da")
    if db is not None:
        want = ad.t() @ dz
        bound = ad.abs().t() @ ez + acc_error(a.dtype, M) * (ad.abs().t() @ (dz.abs() + ez))
        assert_within(db, want, bound * 1.01 + rounding(want, a.dtype), "db")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N,K", SMALL + [(1023, 1025, 17), (513, 640, 320)])
def test_epilogue_backward_sizes(h, M, N, K, dtype):
    t = TYPES[dtype]
    a, b = operands(M, N, K, dtype, 10 * M + N)
    check_epilogue_backward(h, matrix(M, N, t, 4), a, b, matrix(M, N, t, 5), "gelu")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_epilogue_backward_activations(h, dtype, act):
    t = TYPES[dtype]
    a, b = operands(130, 264, 136, dtype, 3)
    pre = matrix(130, 264, t, 5, scale=4.0)
    pre[0, :8] = 0  # relu's corner
    check_epilogue_backward(h, matrix(130, 264, t, 4), a, b, pre, act, bias_dtype="f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("b_layout", ["row", "col"])
@pytest.mark.parametrize("a_layout", ["row", "col"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 1)])
def test_epilogue_backward_layouts(h, a_layout, b_layout, pad, offset, dtype):
    t = TYPES[dtype]
    a, b = operands(260, 200, 136, dtype, 31, a_layout, b_layout, pad, offset)
    dy, pre = matrix(260, 200, t, 4, pad=pad, offset=offset), matrix(260, 200, t, 5, pad=2 * pad)
    check_epilogue_backward(h, dy, a, b, pre, "silu")


def test_epilogue_backward_parts_and_types(h):
    a, b = operands(100, 72, 40, "bf16", 31)
    dy, pre = matrix(100, 72, torch.bfloat16, 4), matrix(100, 72, torch.bfloat16, 5)
    for need in ((True, False, False), (False, True, False), (False, False, True), (False,) * 3):
        check_epilogue_backward(h, dy, a, b, pre, "gelu_tanh", need)
        check_epilogue_backward(h, dy, a, b, None, None, need)
    # a gradient wider than the operands
    check_epilogue_backward(h, dy.float(), a, b, pre.float(), "silu", bias_dtype="f32")
    check_epilogue_backward(h, dy.float(), a, b, None, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_epilogue_backward_empty_extents(h, dtype):
    t = TYPES[dtype]
    e = lambda *s: torch.empty(*s, dtype=t, device="cuda")
    da, db, dbias = h.matmul_epilogue_backward(e(0, 40), e(0, 24), matrix(24, 40, t, 1),
                                               pre=e(0, 40), activation="silu")
    assert da.shape == (0, 24) and (db == 0).all() and (dbias == 0).all()
    da, db, dbias = h.matmul_epilogue_backward(e(5, 0), matrix(5, 24, t, 1), e(24, 0))
    assert (da == 0).all() and db.shape == (24, 0) and dbias.shape == (0,)
    dy = matrix(5, 40, t, 1)
    da, db, dbias = h.matmul_epilogue_backward(dy, e(5, 0), e(0, 40))
    assert da.shape == (5, 0) and db.shape == (0, 40)
    assert_within(dbias, dy.double().sum(0),
                  2.0 ** -19 * dy.double().abs().sum(0) + rounding(dy.double().sum(0), t))


def check_gated_backward(h, dh, x, wg, wu, g, u, act, need=(True, True, True)):
    M, K = x.shape
    F = wg.shape[1]
    dx, dwg, dwu = h.gated_backward(dh, x, wg, wu, g, u, activation=act, need=need)
    torch.cuda.synchronize()
    gd, ud, hd, xd = g.double(), u.double(), dh.double(), x.double()
    dg = hd * ud * slope64(gd, act)
    du = hd * act64(gd, act)
    eg = 2.0 ** -19 * (1 + gd.abs()) * (hd * ud).abs() + rounding(dg, x.dtype)
    eu = 2.0 ** -19 * (1 + gd.abs()) * hd.abs() + rounding(du, x.dtype)
    if dx is not None:
        wgd, wud = wg.double().t(), wu.double().t()
        want = dg @ wgd + du @ wud
        rel = acc_error(x.dtype, 2 * F)
        bound = eg @ wgd.abs() + eu @ wud.abs() + rel * ((dg.abs() + eg) @ wgd.abs() + (
            du.abs() + eu) @ wud.abs())
        assert_within(dx, want, bound * 1.01 + rounding(want, x.dtype), "dx")
    for dw, d, e, what in ((dwg, dg, eg, "dwg"), (dwu, du, eu, "dwu")):
        if dw is not None:
            want = xd.t() @ d
            bound = xd.abs().t() @ e + acc_error(x.dtype, M) * (xd.abs().t() @ (d.abs() + e))
            assert_within(dw, want, bound * 1.01 + rounding(want, x.dtype), what)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,F,K", SMALL + [(1023, 1025, 40), (513, 640, 320), (200, 1000, 1032)])
def test_gated_backward_sizes(h, M, F, K, dtype):
    t = TYPES[dtype]
    x, wg = operands(M, F, K, dtype, 10 * M + F)
    wu = matrix(K, F, t, 9, "col", scale=K ** -0.5)
    check_gated_backward(h, matrix(M, F, t, 4), x, wg, wu, matrix(M, F, t, 5), matrix(M, F, t, 6),
                         "silu")


@pytest.mark.parametrize("act", ACTS)
def test_gated_backward_activations(h, act):
    t = torch.bfloat16
    x, wg = operands(130, 264, 136, "bf16", 3)
    wu = matrix(136, 264, t, 9, "col", scale=0.1)
    check_gated_backward(h, matrix(130, 264, t, 4), x, wg, wu, matrix(130, 264, t, 5, scale=4.0),
                         matrix(130, 264, t, 6), act)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("w_layout", ["row", "col"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (3, 1)])
def test_gated_backward_layouts(h, w_layout, pad, offset, dtype):
    t = TYPES[dtype]
    x, wg = operands(260, 200, 136, dtype, 31, "row", w_layout, pad, offset)
    wu = matrix(136, 200, t, 9, w_layout, pad + 8, offset, scale=0.1)
    both = matrix(260, 400, t, 5, pad=pad, offset=offset)
    dh = matrix(260, 200, t, 4, pad=pad, offset=offset)
    check_gated_backward(h, dh, x, wg, wu, both[:, :200], both[:, 200:], "gelu_tanh")


def test_gated_backward_parts(h):
    t = torch.bfloat16
    x, wg = operands(100, 72, 40, "bf16", 31)
    wu = matrix(40, 72, t, 9, "col", scale=0.1)
    rest = [matrix(100, 72, t, s) for s in (4, 5, 6)]
    for need in ((True, False, False), (False, True, False), (False, False, True), (False,) * 3,
                 (True, False, True)):
        check_gated_backward(h, rest[0], x, wg, wu, rest[1], rest[2], "silu", need)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gated_backward_empty_extents(h, dtype):
    t = TYPES[dtype]
    e = lambda *s: torch.empty(*s, dtype=t, device="cuda")
    w = matrix(24, 40, t, 1, "col")
    dx, dwg, dwu = h.gated_backward(e(0, 40), e(0, 24), w, w, e(0, 40), e(0, 40))
    assert dx.shape == (0, 24) and (dwg == 0).all() and (dwu == 0).all()
    dx, dwg, dwu = h.gated_backward(e(5, 0), matrix(5, 24, t, 1), e(24, 0), e(24, 0), e(5, 0), e(5, 0))
    assert (dx == 0).all() and dwg.shape == (24, 0)


@pytest.mark.parametrize("op", ["epilogue", "gated"])
def test_gradients_against_differences(h, op):
    """<grad, d> against central differences of <c, forward> along random directions d, in
    exact fp32. The third derivatives of silu stay below 1, so with steps of 1e-2 the
    truncation is below 1e-4 of the gradient's size; fp32 forward values good to 1e-6 and a
    step of 1e-2 leave another 1e-4: 1e-3 of |c| |d| with room for the sums."""
    M, N, K = 24, 40, 36
    x = matrix(M, K, torch.float32, 1)
    w = matrix(K, N, torch.float32, 2, "col", scale=K ** -0.5)
    v = matrix(K, N, torch.float32, 3, "col", scale=K ** -0.5)
    bias = matrix(1, N, torch.float32, 7)[0]
    c = matrix(M, N, torch.float32, 4)

    def forward(x, w, v, bias):
        y = (h.matmul_epilogue(x, w, bias=bias, activation="silu") if op == "epilogue"
             else h.gated(x, w, v, activation="silu"))
        return float((y.double() * c.double()).sum())

    if op == "epilogue":
        _, pre = h.matmul_epilogue(x, w, bias=bias, activation="silu", save=True)
        dx, dw, db = h.matmul_epilogue_backward(c, x, w, pre=pre, activation="silu")
        grads = [dx, dw, None, db]
    else:
        _, g, u = h.gated(x, w, v, activation="silu", save=True)
        grads = list(h.gated_backward(c, x, w, v, g, u, activation="silu")) + [None]
    step = 1e-2
    for k, grad in enumerate(grads):
        if grad is None:
            continue
        args = [x, w, v, bias]
        d = torch.randn(args[k].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(k))
        hi, lo = list(args), list(args)
        hi[k], lo[k] = args[k] + step * d, args[k] - step * d
        hi, lo = [[t if i == 3 else t if i == 0 else t.t().contiguous().t()
                   for i, t in enumerate(v)] for v in (hi, lo)]
        slope = (forward(*hi) - forward(*lo)) / (2 * step)
        want = float((grad.double() * d.double()).sum())
        size = float(grad.double().norm()) * float(d.double().norm())
        assert abs(slope - want) <= 1e-3 * size, (k, slope, want, size)


# ------------------------------------------------------------ streams, graphs, refusals

def test_calls_repeat_bit_for_bit_and_on_another_stream(h):
    x, wg = operands(300, 264, 1024, "bf16", 3)
    wu = matrix(1024, 264, torch.bfloat16, 9, "col", scale=0.03)
    xs = x[:5].contiguous()
    dh = matrix(300, 264, torch.bfloat16, 4)
    first = [*h.gated(x, wg, wu, save=True), h.gated(xs, wg, wu), h.matmul_epilogue(xs, wg)]
    grads = h.gated_backward(dh, x, wg, wu, first[1], first[2])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        again = [*h.gated(x, wg, wu, save=True), h.gated(xs, wg, wu), h.matmul_epilogue(xs, wg)]
        again += h.gated_backward(dh, x, wg, wu, again[1], again[2])
    s.synchronize()
    for p, q in zip(first + list(grads), again):
        assert torch.equal(p, q)


def test_graph_replay(h):
    """Captured calls replay on new values in the same buffers."""
    x, w = operands(1, 512, 1024, "bf16", 3)
    r = matrix(1, 512, torch.bfloat16, 6)
    x2, w2 = operands(300, 264, 128, "bf16", 4)
    calls = lambda: (h.matmul_epilogue(x, w, activation="gelu", residual=r),
                     h.gated(x2, w2, w2, save=False))
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        calls()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y, y2 = calls()
    for seed in (50, 60):
        x.copy_(matrix(1, 1024, torch.bfloat16, seed))
        x2.copy_(matrix(300, 128, torch.bfloat16, seed))
        graph.replay()
        torch.cuda.synchronize()
        e, e2 = calls()
        assert torch.equal(y, e) and torch.equal(y2, e2)


def test_refusals(h):
    import dense_tiled_gemm_05_gb300 as g
    t = torch.bfloat16
    a, b = matrix(8, 32, t, 1), matrix(32, 16, t, 2)
    with pytest.raises(ValueError):
        h.matmul_epilogue(a, matrix(31, 16, t, 2))
    with pytest.raises(TypeError):
        h.matmul_epilogue(a, b.float())
    with pytest.raises(ValueError):
        h.matmul_epilogue(a, b, activation="tanh")
    with pytest.raises(ValueError):
        h.matmul_epilogue(a, b, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(ValueError):
        h.matmul_epilogue(a, b, residual=matrix(8, 15, t, 1))
    with pytest.raises(TypeError):
        h.matmul_epilogue(a, b, residual=matrix(8, 16, torch.float32, 1))
    with pytest.raises(ValueError):
        h.matmul_epilogue(a, b, residual=matrix(8, 16, t, 1, "col"))
    with pytest.raises(ValueError):
        h.matmul_epilogue(a.cpu(), b.cpu())
    with pytest.raises(TypeError):
        h.matmul_epilogue(a, b, bias=torch.zeros(16, dtype=torch.int32, device="cuda"))
    for kw, status in ((dict(precision="tf32"), "GEMM_ERR_UNSUPPORTED"),
                       (dict(out=a[:, :16]), "GEMM_ERR_INVALID_ARG")):
        with pytest.raises(g.GemmError) as e:
            h.matmul_epilogue(a, b, activation="silu", **kw)
        assert e.value.status == status
    store = torch.zeros(9, 16, dtype=t, device="cuda")
    with pytest.raises(g.GemmError):  # the residual half over the output
        h.matmul_epilogue(a, b, residual=store[1:], out=store[:8])
    with pytest.raises(ValueError):
        h.matmul_epilogue_backward(matrix(8, 16, t, 3), a, b, activation="silu")
    with pytest.raises(ValueError):
        h.matmul_epilogue_backward(matrix(8, 15, t, 3), a, b)
    with pytest.raises(ValueError):
        h.gated(a, b, matrix(32, 15, t, 2))
    with pytest.raises(ValueError):
        h.gated(a, b, matrix(32, 16, t, 2, "col"))
    with pytest.raises(g.GemmError):
        h.gated(a, b, b, out=a[:, :16])
    with pytest.raises(g.GemmError) as e:
        h.gated(a.half(), b.half(), b.half(), precision="f16acc")
    assert e.value.status == "GEMM_ERR_UNSUPPORTED"
    with pytest.raises(TypeError):
        h.gated_backward(matrix(8, 16, torch.float32, 3), a, b, b, *[matrix(8, 16, t, 3)] * 2)
    # the C entries' own checks
    L = g.lib()
    p = a.data_ptr()
    args = lambda **k: [h.handle, 8, 16, 32, p, 32, b.data_ptr(), 16, store.data_ptr(), 16, 2, 2,
                        0, 0, 0]
    ep = g.Epilogue()
    ep.activation = 9
    assert L.gemm_run_epilogue(*args(), ep, None) == 1
    ep.activation, ep.bias, ep.bias_dtype = 0, store.data_ptr() + 1, 2
    assert L.gemm_run_epilogue(*args(), ep, None) == 3
    ep.bias, ep.pre, ep.ld_pre = None, store.data_ptr(), 16
    assert L.gemm_run_epilogue(*args(), ep, None) == 1  # pre over C
    ep.ld_pre = 15
    assert L.gemm_run_epilogue(*args(), ep, None) == 1
    assert h.status() == 0
