"""Feed-forward operators on elements more than 2^32 (of a matrix with a long leading dimension) and
2^31 (of a dense one) from a matrix's first: offsets that 32-bit arithmetic would wrap."""
import pytest
import torch

from ff_util import TYPES, acc_error, act64, assert_within, matrix, rounding, slope64
from test_feed_forward_gpu import (check_epilogue, check_epilogue_backward, check_gated,
                                   check_gated_backward)
from test_layer_norm_gpu import check_backward, check_norm, saved, stats

pytestmark = pytest.mark.gpu


@pytest.fixture()
def h():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    if torch.cuda.mem_get_info()[0] < 200 << 30:
        pytest.skip("needs 200 GB")
    import dense_tiled_gemm_05_gb300 as g
    hh = g.Gemm(0)
    yield hh
    assert hh.status() == 0
    hh.close()
    torch.cuda.empty_cache()


def far(rows, cols, t, seed, aligned=True):
    """A rows x cols view whose last row starts 2^32 elements into its buffer."""
    ld = -(-(1 << 32) // (rows - 1)) // 8 * 8 + (8 if aligned else 9)
    view = torch.empty((rows - 1) * ld + cols, dtype=t, device="cuda").as_strided((rows, cols), (ld, 1))
    assert (rows - 1) * ld >= 1 << 32
    view.copy_(matrix(rows, cols, t, seed))
    return view


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_epilogue(h, M, dtype, aligned):
    t = TYPES[dtype]
    a, w = far(M, 200, t, 1, aligned), far(264, 200, t, 2, aligned)
    r, out = far(M, 264, t, 3, aligned), far(M, 264, t, 4, aligned)
    check_epilogue(h, a, w.t(), "silu", None, r, out=out, save=False)
    check_epilogue(h, a, w.t(), None, None, r, out=r, save=False)
    check_epilogue_backward(h, out, a, w.t(), r, "silu")


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_gated(h, M, dtype, aligned):
    t = TYPES[dtype]
    x, wg, wu = far(M, 200, t, 1, aligned), far(264, 200, t, 2, aligned), far(264, 200, t, 3, aligned)
    wg *= 0.07
    wu *= 0.07
    check_gated(h, x, wg.t(), wu.t(), "silu", save=True)
    dh, g, u = (far(M, 264, t, s, aligned) for s in (4, 5, 6))
    check_gated_backward(h, dh, x, wg.t(), wu.t(), g, u, "silu")


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_tensor_core_kernels_and_unfused(h, M, aligned):
    a, w = far(M, 200, torch.bfloat16, 1, aligned), far(264, 200, torch.bfloat16, 2, aligned)
    r, out = (far(M, 264, torch.bfloat16, s, aligned) for s in (3, 4))
    for pair in (1, 2):
        h.set_option("cta_pair", pair)
        check_epilogue(h, a, w.t(), "gelu", None, r, out=out, save=True)
    h.set_option("cta_pair", 0)
    a, w, r, out = a.float(), w.float(), None, None
    r, out = far(M, 264, torch.float32, 3, aligned), far(M, 264, torch.float32, 4, aligned)
    check_epilogue(h, a, w.t(), "gelu", None, r, out=out, save=True, precision="tf32")


@pytest.mark.parametrize("aligned", [True, False])
@pytest.mark.parametrize("M,N", [(40, 1000), (40, 9000), (40, 20000), (1300, 1000)])
def test_layer_norm(h, M, N, aligned):
    x, out = far(M, N, torch.bfloat16, 1, aligned), far(M, N, torch.bfloat16, 2, aligned)
    w = matrix(1, N, torch.float32, 3)[0]
    check_norm(h, x, w, None, out=out)
    check_backward(h, out, x, w, *saved(x))
    check_backward(h, far(M, N, torch.float32, 5, aligned), x, w, *saved(x))


def sample(M, N):
    """Rows at both ends and where the offset passes 2^31."""
    mid = (1 << 31) // N
    return torch.tensor([0, 1, mid - 1, mid, mid + 1, M - 2, M - 1], device="cuda")


def rows_of(M, N, t, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(M, N, generator=gen, device="cuda", dtype=t)


@pytest.mark.parametrize("M,N", [(270000, 8192), (2200000, 1001)])
def test_dense_layer_norm(h, M, N):
    t = torch.bfloat16
    x, w = rows_of(M, N, t, 1), matrix(1, N, torch.float32, 3)[0]
    y, mean, rstd = h.layer_norm(x, w, None, save=True)
    i = sample(M, N)
    m, r = stats(x[i].double(), 1e-5)
    want = (x[i].double() - m) * r * w.double()
    assert_within(y[i], want, 2.0 ** -17 * (want.abs() + w.double().abs()) + rounding(want, t), "y")
    dy = rows_of(M, N, t, 2)
    dx, dw, db = h.layer_norm_backward(dy, x, w, mean, rstd)
    m, r = mean[i, None].double(), rstd[i, None].double()
    xh, v = (x[i].double() - m) * r, dy[i].double() * w.double()
    want = r * (v - v.mean(1, keepdim=True) - xh * (v * xh).mean(1, keepdim=True))
    assert_within(dx[i], want, 2.0 ** -17 * (v.abs() + xh.abs() + 1) + rounding(want, t), "dx")
    # the sums over all rows: magnitudes of about 0.8 a term, fp32 sums of some hundred rows and
    # a tree of bands
    sw = sb = 0
    for k in range(0, M, 100000):
        d = dy[k:k + 100000].double()
        sb = sb + d.sum(0)
        sw = sw + (d * (x[k:k + 100000].double() - mean[k:k + 100000, None]) * rstd[k:k + 100000, None]).sum(0)
    bound = torch.full_like(sb, M * 2.0 ** -12 * 2.0 ** -8)
    assert_within(db, sb, bound, "db")
    assert_within(dw, sw, bound, "dw")


@pytest.mark.parametrize("F", [66000, 66001])
def test_dense_gated_training(h, F):
    """2^31 elements of h, twice as many of the kept products and of their gradients."""
    M, K, t = 33000, 64, torch.bfloat16
    x, wg, wu = rows_of(M, K, t, 1), rows_of(F, K, t, 2) * 0.125, rows_of(F, K, t, 3) * 0.125
    out, g, u = h.gated(x, wg.t(), wu.t(), save=True)
    i = sample(M, F)
    for kept, w in ((g, wg), (u, wu)):
        want = x[i].double() @ w.t().double()
        e = acc_error(t, K) * (x[i].double().abs() @ w.t().double().abs())
        assert_within(kept[i], want, e + rounding(want, t), "kept")
    want = act64(x[i].double() @ wg.t().double(), "silu") * (x[i].double() @ wu.t().double())
    assert_within(out[i], want, 2.0 ** -14 * (want.abs() + 1) + rounding(want, t), "h")
    dh = out  # (any values)
    dx, dwg, dwu = h.gated_backward(dh, x, wg.t(), wu.t(), g, u)
    gd, ud, hd = g[i].double(), u[i].double(), dh[i].double()
    dg, du = hd * ud * slope64(gd, "silu"), hd * act64(gd, "silu")
    want = dg @ wg.double() + du @ wu.double()
    size = dg.abs() @ wg.double().abs() + du.abs() @ wu.double().abs()
    assert_within(dx[i], want, 2.0 ** -8 * size + rounding(want, t), "dx")
    j = torch.tensor([0, 1, F // 2, F - 2, F - 1], device="cuda")
    gd, ud, hd = g[:, j].double(), u[:, j].double(), dh[:, j].double()
    for got, d in ((dwg, hd * ud * slope64(gd, "silu")), (dwu, hd * act64(gd, "silu"))):
        want = x.double().t() @ d
        size = x.double().abs().t() @ d.abs()
        assert_within(got[:, j], want, 2.0 ** -8 * size + rounding(want, t), "dw")


@pytest.mark.parametrize("N", [66000, 66001])
def test_dense_epilogue_training(h, N):
    M, K, t = 33000, 64, torch.bfloat16
    x, w, r = rows_of(M, K, t, 1), rows_of(N, K, t, 2) * 0.125, rows_of(M, N, t, 3)
    y, z = h.matmul_epilogue(x, w.t(), activation="gelu", residual=r, save=True)
    i = sample(M, N)
    want = x[i].double() @ w.t().double()
    e = acc_error(t, K) * (x[i].double().abs() @ w.t().double().abs())
    assert_within(z[i], want, e + rounding(want, t), "pre")
    want = act64(want, "gelu") + r[i].double()
    assert_within(y[i], want, 2 * e + 2.0 ** -18 * (want.abs() + 1) + rounding(want, t), "y")
    da, db, dbias = h.matmul_epilogue_backward(r, x, w.t(), pre=z, activation="gelu", bias_dtype="f32")
    dz = r[i].double() * slope64(z[i].double(), "gelu")
    want, size = dz @ w.double(), dz.abs() @ w.double().abs()
    assert_within(da[i], want, 2.0 ** -8 * size + rounding(want, t), "da")
    j = torch.tensor([0, 1, N // 2, N - 2, N - 1], device="cuda")
    dz = r[:, j].double() * slope64(z[:, j].double(), "gelu")
    want, size = x.double().t() @ dz, x.double().abs().t() @ dz.abs()
    assert_within(db[:, j], want, 2.0 ** -8 * size + rounding(want, t), "db")
    assert_within(dbias[j], dz.sum(0), 2.0 ** -17 * dz.abs().sum(0), "dbias")
