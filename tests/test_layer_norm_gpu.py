"""Layer norm and its backward pass on the GPU against their definitions in 64 bits: every
row-length class of the kernels, odd widths, each type, padded and misaligned rows, large
offsets and tiny variances, and the refusals."""
import itertools

import pytest
import torch

from ff_util import TYPES, assert_within, matrix, rounding

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 64), (4, 130), (9, 513), (1000, 96), (33, 1025),
          (64, 2048), (300, 1000), (17, 4095), (40, 5000), (12, 8192), (7, 12288), (5, 16385),
          (3, 33000), (2, 70001)]


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    hh = g.Gemm(0)
    yield hh
    hh.close()


def stats(x, eps):
    mean = x.mean(1, keepdim=True)
    return mean, 1 / torch.sqrt((x - mean).square().mean(1, keepdim=True) + eps)


def sums(N):
    """Relative error of a sum over N values of a row (see ff_util): at most N / 32 of them in
    one thread."""
    return (N / 32 + 32) * 2.0 ** -24


def check_norm(h, x, w, b, eps=1e-5, out_dtype=None, out=None):
    M, N = x.shape
    xd = x.double()
    got, mean, rstd = h.layer_norm(x, w, b, eps=eps, out=out, out_dtype=out_dtype, save=True)
    torch.cuda.synchronize()
    m, r = stats(xd, eps)
    e_mean = sums(N) * xd.abs().mean(1, keepdim=True) + 2.0 ** -24 * m.abs()
    assert_within(mean[:, None], m, e_mean, "mean")
    # the variance's own sum, the centring's rounding, and the mean's error
    e_d = e_mean + 2.0 ** -23 * (xd.abs() + m.abs())
    dd = (xd - m).abs()
    e_var = sums(N) * dd.square().mean(1, keepdim=True) + (2 * dd * e_d + e_d * e_d).mean(
        1, keepdim=True)
    e_r = 0.5 * r ** 3 * e_var * (1 + 2 * r * r * e_var) + 2.0 ** -21 * r
    assert_within(rstd[:, None], r, e_r, "rstd")
    wd = torch.ones(N, dtype=torch.float64, device="cuda") if w is None else w.double()
    bd = 0 if b is None else b.double()
    want = (xd - m) * r * wd + bd
    bound = wd.abs() * (e_d * r + (dd + e_d) * e_r) + 2.0 ** -22 * (want.abs() + (dd * r * wd).abs())
    assert_within(got, want, 1.01 * bound + rounding(want, got.dtype), "y")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_norm_sizes(h, M, N, dtype):
    x = matrix(M, N, TYPES[dtype], M + N) * 2 + 0.5
    p = torch.float32 if N % 2 else TYPES[dtype]
    check_norm(h, x, matrix(1, N, p, 2)[0], matrix(1, N, p, 3)[0])


@pytest.mark.parametrize("in_dtype,param,out_dtype", list(itertools.product(TYPES, repeat=3)))
def test_norm_types(h, in_dtype, param, out_dtype):
    x = matrix(20, 1000, TYPES[in_dtype], 4)
    check_norm(h, x, matrix(1, 1000, TYPES[param], 2)[0], matrix(1, 1000, TYPES[param], 3)[0],
               out_dtype=out_dtype)


@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 1)])
@pytest.mark.parametrize("N", [40, 1000, 1001, 8200])
def test_norm_padded_rows(h, N, pad, offset):
    for dtype in ("bf16", "f32"):
        t = TYPES[dtype]
        x = matrix(11, N, t, 4, pad=pad, offset=offset)
        store = torch.full((11, N + 5), 7.0, dtype=t, device="cuda")
        w = matrix(1, N + 1, t, 2)[0][1:]
        check_norm(h, x, w, None, out=store[:, :N])
        assert (store[:, N:] == 7).all()
        check_norm(h, x, None, w)


def test_norm_in_place_and_without_parameters(h):
    for N in (100, 5000, 40000):
        x = matrix(6, N, torch.float32, 4)
        want = h.layer_norm(x)
        y = h.layer_norm(x, out=x)
        assert y.data_ptr() == x.data_ptr() and torch.equal(y, want)
        check_norm(h, matrix(6, N, torch.float32, 4), None, None)


def test_norm_offsets_and_flat_rows(h):
    """A mean far larger than the spread, equal values in a row (rstd is 1 / sqrt(eps)), and
    special values."""
    x = matrix(4, 1000, torch.float32, 4) * 1e-2 + 1000.0
    x[1] = 3.0
    x[2] = 0.0
    check_norm(h, x, None, None)
    y, mean, rstd = h.layer_norm(x, eps=0.25, save=True)
    assert (y[1:3] == 0).all() and (mean[1:3].cpu() == torch.tensor([3.0, 0.0])).all()
    assert (rstd[1:3] == 2.0).all()
    x[3, 7] = float("inf")
    x[0, 3] = float("nan")
    y = h.layer_norm(x)
    assert torch.isnan(y[0]).all() and torch.isnan(y[3]).all() and torch.isfinite(y[1:3]).all()


def check_backward(h, dy, x, w, mean, rstd, need=(True, True, True), param_dtype=None):
    M, N = x.shape
    dx, dw, db = h.layer_norm_backward(dy, x, w, mean, rstd, need=need, param_dtype=param_dtype)
    torch.cuda.synchronize()
    m, r = mean.double()[:, None], rstd.double()[:, None]
    xd, d = x.double(), dy.double()
    wd = torch.ones(N, dtype=torch.float64, device="cuda") if w is None else w.double()
    xh = (xd - m) * r
    # errors of xh: the difference's and the product's roundings
    size = (xd - m).abs() * r * (1 + 2.0 ** -20)
    v = d * wd
    a, b = v.mean(1, keepdim=True), (v * xh).mean(1, keepdim=True)
    if dx is not None:
        want = r * (v - a - xh * b)
        e = 2 * sums(N)
        bound = r * (e * v.abs().mean(1, keepdim=True) + size * e * (v.abs() * size).mean(
            1, keepdim=True) + 2.0 ** -21 * (v.abs() + a.abs() + size * b.abs()))
        assert_within(dx, want, bound + rounding(want, dx.dtype), "dx")
    e = (M + 32) * 2.0 ** -24 + 2.0 ** -22
    if dw is not None:
        want = (d * xh).sum(0)
        assert_within(dw, want, e * (d.abs() * size).sum(0) + rounding(want, dw.dtype), "dw")
    if db is not None:
        want = d.sum(0)
        assert_within(db, want, e * d.abs().sum(0) + rounding(want, db.dtype), "db")


def saved(x, eps=1e-5):
    m, r = stats(x.double(), eps)
    return m[:, 0].float(), r[:, 0].float()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_norm_backward_sizes(h, M, N, dtype):
    t = TYPES[dtype]
    x = matrix(M, N, t, M + N) * 2 + 0.5
    p = torch.float32 if N % 2 else t
    check_backward(h, matrix(M, N, t, 5), x, matrix(1, N, p, 2)[0], *saved(x))


@pytest.mark.parametrize("in_dtype,param,out_dtype", list(itertools.product(TYPES, repeat=3)))
def test_norm_backward_types(h, in_dtype, param, out_dtype):
    x = matrix(20, 1000, TYPES[in_dtype], 4)
    check_backward(h, matrix(20, 1000, TYPES[out_dtype], 5), x,
                   matrix(1, 1000, TYPES[param], 2)[0], *saved(x))


@pytest.mark.parametrize("pad,offset", [(8, 8), (3, 1)])
@pytest.mark.parametrize("N", [40, 1000, 1001, 8200])
def test_norm_backward_padded_rows(h, N, pad, offset):
    for dtype in ("bf16", "f32"):
        t = TYPES[dtype]
        x = matrix(70, N, t, 4, pad=pad, offset=offset)
        dy = matrix(70, N, t, 5, pad=2 * pad, offset=offset)
        check_backward(h, dy, x, matrix(1, N + 1, t, 2)[0][1:], *saved(x))


def test_norm_backward_parts(h):
    x, dy = matrix(50, 264, torch.bfloat16, 4), matrix(50, 264, torch.bfloat16, 5)
    w = matrix(1, 264, torch.float32, 2)[0]
    for need in itertools.product((True, False), repeat=3):
        check_backward(h, dy, x, w, *saved(x), need=need)
        check_backward(h, dy, x, None, *saved(x), need=need, param_dtype="bf16")


def test_norm_backward_repeats_bit_for_bit(h):
    x, dy = matrix(3000, 1000, torch.bfloat16, 4), matrix(3000, 1000, torch.bfloat16, 5)
    w = matrix(1, 1000, torch.float32, 2)[0]
    first = h.layer_norm_backward(dy, x, w, *saved(x))
    for _ in range(3):
        for p, q in zip(first, h.layer_norm_backward(dy, x, w, *saved(x))):
            assert torch.equal(p, q)


def test_norm_empty_extents(h):
    e = lambda *s: torch.empty(*s, dtype=torch.float32, device="cuda")
    assert h.layer_norm(e(0, 40)).shape == (0, 40)
    assert h.layer_norm(e(4, 0)).shape == (4, 0)
    dx, dw, db = h.layer_norm_backward(e(0, 40), e(0, 40), None, e(0), e(0))
    assert dx.shape == (0, 40) and (dw == 0).all() and (db == 0).all()
    dx, dw, db = h.layer_norm_backward(e(4, 0), e(4, 0), None, e(4), e(4))
    assert dx.shape == (4, 0) and dw.shape == (0,)


def test_norm_gradients_against_differences(h):
    """<grad, d> against central differences of <c, y> in fp32: steps of 1e-2 against values
    of order 1 leave 1e-4 of truncation and, with y good to 1e-6, 1e-4 of rounding."""
    M, N = 12, 200
    x, c = matrix(M, N, torch.float32, 1), matrix(M, N, torch.float32, 2)
    w, b = matrix(1, N, torch.float32, 3)[0], matrix(1, N, torch.float32, 4)[0]
    _, mean, rstd = h.layer_norm(x, w, b, save=True)
    grads = h.layer_norm_backward(c, x, w, mean, rstd)
    step = 1e-2
    for k in range(3):
        args = [x, w, b]
        d = torch.randn(args[k].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(k))
        val = []
        for sign in (1, -1):
            moved = list(args)
            moved[k] = args[k] + sign * step * d
            val.append(float((h.layer_norm(*moved).double() * c.double()).sum()))
        want = float((grads[k].double() * d.double()).sum())
        size = float(grads[k].double().norm()) * float(d.double().norm())
        assert abs((val[0] - val[1]) / (2 * step) - want) <= 1e-3 * size, k


def test_norm_refusals(h):
    import dense_tiled_gemm_05_gb300 as g
    x = matrix(4, 64, torch.float32, 1)
    w = torch.ones(64, device="cuda")
    with pytest.raises(ValueError):
        h.layer_norm(x.t())
    with pytest.raises(ValueError):
        h.layer_norm(x, torch.ones(63, device="cuda"))
    with pytest.raises(ValueError):
        h.layer_norm(x.cpu())
    with pytest.raises(TypeError):
        h.layer_norm(x, w, w.half())
    with pytest.raises(TypeError):
        h.layer_norm(x.double())
    for eps in (-1.0, float("nan"), float("inf")):
        with pytest.raises(g.GemmError):
            h.layer_norm(x, eps=eps)
    with pytest.raises(g.GemmError):  # rows shifted over one another
        h.layer_norm(x[:3], out=x[1:])
    mean, rstd = saved(x)
    with pytest.raises(TypeError):
        h.layer_norm_backward(x, x, w, mean.double(), rstd)
    with pytest.raises(ValueError):
        h.layer_norm_backward(x, x, w, mean[:3], rstd)
    with pytest.raises(ValueError):
        h.layer_norm_backward(x[:3], x, w, mean, rstd)
    L = g.lib()
    p = x.data_ptr()
    q = torch.empty_like(x).data_ptr()
    run = lambda *a: L.gemm_layer_norm(h.handle, *a, None)
    assert run(4, 64, p, 63, 0, 0, q, 64, 0, 0, 1e-5, 0, 0, 0) == 1   # ldx below N
    assert run(4, 64, p + 2, 64, 0, 0, q, 64, 0, 0, 1e-5, 0, 0, 0) == 3
    assert run(4, 64, 0, 64, 0, 0, q, 64, 0, 0, 1e-5, 0, 0, 0) == 1
    assert run(-1, 64, p, 64, 0, 0, q, 64, 0, 0, 1e-5, 0, 0, 0) == 1
    assert run(4, 64, p, 64, 0, 0, q, 64, 0, 0, 1e-5, 5, 0, 0) == 1
    assert L.gemm_layer_norm(None, 4, 64, p, 64, 0, 0, q, 64, 0, 0, 1e-5, 0, 0, 0, None) == 1
    assert h.status() == 0
