"""Row counts at which every group of threads of the feed-forward operators' row kernels walks
several rows: the layer norm's wide kernel (taken from eight rows an SM on), its backward pass, and
the slopes and column sums, against their definitions in 64 bits."""
import pytest
import torch

from ff_util import TYPES, matrix
from test_feed_forward_gpu import (check_epilogue, check_epilogue_backward, check_gated,
                                   check_gated_backward)
from test_layer_norm_gpu import check_backward, check_norm, saved

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def h():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    hh = g.Gemm(0)
    yield hh
    assert hh.status() == 0
    hh.close()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# columns and the groups an SM runs at once there: 32 threads a row up to 1024 columns, ... 512
# threads from 8193 on (1024 threads an SM; one CTA of 512 for the widest)
WIDE = [(264, 32), (1000, 32), (1024, 32), (1032, 16), (2000, 16), (2056, 8), (4096, 8), (4104, 4),
        (8192, 4), (8200, 2), (16384, 2)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,groups", WIDE)
def test_norm(h, N, groups, dtype):
    """Three and a half rows a group, and a row more: every stage of the ring is used again, and
    the groups end apart."""
    t = TYPES[dtype]
    M = sms() * max(groups * 7 // 2, 8) + 1
    x = matrix(M, N, t, 4) * 2 + 0.5
    p = torch.float32 if N % 16 else t
    check_norm(h, x, matrix(1, N, p, 2)[0], matrix(1, N, p, 3)[0])


@pytest.mark.parametrize("N", [264, 4096, 8200])
def test_norm_in_place_and_padded(h, N):
    M = sms() * 120 + 1 if N == 264 else sms() * 20 + 3
    x = matrix(M, N, torch.bfloat16, 4, pad=8, offset=8)
    want = h.layer_norm(x)
    check_norm(h, x, None, None)
    y = h.layer_norm(x, out=x)
    assert y.data_ptr() == x.data_ptr() and torch.equal(y, want)


def test_norm_other_output_types(h):
    x = matrix(sms() * 70 + 1, 520, torch.bfloat16, 4)
    w, b = matrix(1, 520, torch.float16, 2)[0], matrix(1, 520, torch.float16, 3)[0]
    for out in ("f32", "f16"):
        check_norm(h, x, w, b, out_dtype=out)


# columns and groups an SM in the backward pass: 16 columns a thread, 512 threads an SM
BACK = [(264, 16), (512, 16), (520, 8), (1000, 8), (1032, 4), (2048, 4), (2056, 2), (4096, 2),
        (4104, 1), (8192, 1), (1001, 8), (4097, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,groups", BACK)
def test_norm_backward(h, N, groups, dtype):
    t = TYPES[dtype]
    M = sms() * groups * 7 // 2 + 1
    x = matrix(M, N, t, 4) * 2 + 0.5
    p = torch.float32 if N % 16 else t
    check_backward(h, matrix(M, N, t, 5), x, matrix(1, N, p, 2)[0], *saved(x))


@pytest.mark.parametrize("grad,N", [("f32", 1000), ("f32", 1001), ("bf16", 9000), ("bf16", 8193)])
def test_norm_backward_two_kernels(h, grad, N):
    """dy of another type, or rows past 8192 columns: several rows a warp in both kernels."""
    M = sms() * 8 * 32 * 2 + 5 if N < 2000 else 3001
    x = matrix(M, N, torch.bfloat16, 4)
    check_backward(h, matrix(M, N, TYPES[grad], 5), x, matrix(1, N, torch.float32, 2)[0], *saved(x))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("F", [264, 520, 257])
def test_slopes(h, F, dtype):
    """About 1520 CTAs of eight rows and 256 columns each: their second and third rows."""
    t = TYPES[dtype]
    M = 1520 * 8 * 5 // 2 // ((F + 255) // 256) + 3
    x, wg, wu = matrix(M, 40, t, 1), *(matrix(40, F, t, s, "col", scale=0.15) for s in (2, 3))
    dy, z, u = (matrix(M, F, t, s) for s in (4, 5, 6))
    check_epilogue_backward(h, dy, x, wg, z, "gelu")
    check_gated_backward(h, dy, x, wg, wu, z, u, "silu")


@pytest.mark.parametrize("F", [264, 257])
def test_rows_after_a_product(h, F):
    """The products that keep their sums in fp32 first (tf32 with an epilogue, and the pair)."""
    t = torch.float32
    M = 1520 * 8 * 5 // 2 // 2 + 3
    x, wg, wu = matrix(M, 40, t, 1), *(matrix(40, F, t, s, "col", scale=0.15) for s in (2, 3))
    r = matrix(M, F, t, 4)
    check_epilogue(h, x, wg, "gelu", matrix(1, F, t, 5)[0], r, precision="tf32")
    check_epilogue(h, x, wg, None, None, r, precision="tf32", out=r, save=False)
    check_gated(h, x, wg, wu, "silu", save=True, precision="tf32")
    check_gated(h, x, wg, wu, "silu", save=False, precision="tf32")
