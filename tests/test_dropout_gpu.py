"""Dropout from a counter: the mask against Philox in numpy, the values against 64 bits."""
import pytest
import torch

from expert_util import kept, philox
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


def key(seed, offset):
    signed = [v - 2 ** 64 if v >= 2 ** 63 else v for v in (seed, offset)]
    return torch.tensor(signed, dtype=torch.int64, device="cuda")


SHAPES = [(1, 1), (1, 4096), (3, 7), (5, 8), (9, 255), (17, 256), (33, 264), (1023, 1025), (300, 2048),
          (2, 20001)]


@pytest.mark.parametrize("M,N", SHAPES)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
def test_values(h, M, N, dtype, pad, offset):
    t, p, seed, call = TYPES[dtype], 0.3, 2 ** 64 - 12345, 2 ** 63 + 77
    x, res = (matrix(M, N, t, s, pad=pad, offset=offset) for s in (1, 2))
    mask, scale = kept(M, N, p, seed, call)
    want = torch.where(mask.cuda(), x.double() * scale, torch.zeros((), dtype=torch.float64, device="cuda"))
    y = h.dropout(x, p, key(seed, call))
    # the scale, the product and (below) the sum are rounded in fp32
    bound = 2.0 ** -23 * want.abs()
    assert y.dtype == t
    assert_within(y, want, bound + rounding(want, t) * (1 + 2.0 ** -23), "dropout")
    assert torch.equal(h.dropout_backward(x, p, key(seed, call)), y)
    total = want + res.double()
    bound = bound + 2.0 ** -24 * total.abs()
    bound = bound + rounding(total, t) * (1 + 2.0 ** -22) + rounding(bound, t)
    y = h.dropout(x, p, key(seed, call), residual=res)
    assert_within(y, total, bound, "dropout with a residual")
    out = x.clone() if not pad and not offset else x
    again = h.dropout(out, p, key(seed, call), residual=res, out=out)
    assert again is out and torch.equal(out, y)
    if not pad and not offset:
        assert torch.equal(h.dropout(x, p, key(seed, call), residual=res, out=res), y)


def test_same_mask_for_every_form(h):
    """The mask is a matter of the place alone: of any type, stride and alignment."""
    M, N = 70, 1000
    k = key(5, 6)
    masks = []
    for dtype in TYPES.values():
        for pad, offset in ((0, 0), (8, 8), (1, 3)):
            x = matrix(M, N, dtype, 1, pad=pad, offset=offset)
            x.fill_(1.0)
            masks.append(h.dropout(x, 0.5, k) != 0)
    assert all(torch.equal(masks[0], m) for m in masks[1:])
    assert not torch.equal(masks[0], h.dropout(torch.ones(M, N, device="cuda"), 0.5, key(5, 7)) != 0)
    assert not torch.equal(masks[0], h.dropout(torch.ones(M, N, device="cuda"), 0.5, key(4, 6)) != 0)


def test_generator():
    """The published answers of Philox4x32-10 for counters and keys of 0s, of 1s and of pi."""
    def words(c, seed):
        return [int(w) for w in philox(c[0], c[1], c[2] | c[3] << 32, seed)]
    ones = 0xFFFFFFFF
    assert words((0, 0, 0, 0), 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert words((ones,) * 4, 2 ** 64 - 1) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    pi = (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344)
    assert words(pi, 0xA4093822 | 0x299F31D0 << 32) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]


@pytest.mark.parametrize("p", [0.0, 1e-6, 0.05, 0.5, 0.9, 0.99999])
def test_share_and_scale(h, p):
    n = 4096
    q = int(p * 65536 + 0.5)
    y = h.dropout(torch.ones(n, n, device="cuda"), p, key(11, 12))
    share = float((y != 0).double().mean())
    keep = 1 - q / 65536
    assert abs(share - keep) <= 5 * (keep * (1 - keep) / n / n) ** 0.5  # five standard deviations
    values = y[y != 0].unique()
    assert len(values) == 1 and abs(float(values[0]) * keep - 1) <= 2.0 ** -23
    if q == 0:
        x = matrix(64, 512, torch.bfloat16, 1)
        assert torch.equal(h.dropout(x, p, key(1, 2)), x)


def test_dropped_elements_leave_nothing(h):
    """NaN and infinities where the mask drops are gone; where it keeps they stay."""
    M, N = 64, 300
    mask = kept(M, N, 0.5, 3, 4)[0].cuda()
    x = torch.where(mask, torch.ones((), device="cuda"), torch.full((), float("nan"), device="cuda"))
    x[0] = float("inf")
    y = h.dropout(x, 0.5, key(3, 4))
    assert torch.equal(torch.isinf(y[0]), mask[0]) and not torch.isnan(y).any()
    assert torch.equal(y[1:] == 2.0, mask[1:])


def test_gradient_against_differences(h):
    """Dropout is linear: the difference of two calls, a step of 1 apart, is the slope."""
    x, k = matrix(6, 50, torch.float32, 5), key(21, 22)
    slope = h.dropout_backward(torch.ones_like(x), 0.25, k)
    up, down = h.dropout(x + 1, 0.25, k), h.dropout(x - 1, 0.25, k)
    assert_within((up - down) / 2, slope.double(), 2.0 ** -21 * (x.double().abs() + 1), "slope")


def test_captured_with_a_new_key(h):
    x, k = torch.ones(100, 512, device="cuda"), key(31, 0)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        y = h.dropout(x, 0.5, k)
        k[1:] += 1
    torch.cuda.synchronize()
    for call in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y != 0, kept(100, 512, 0.5, 31, call)[0].cuda())


def test_rows_past_32_bits(h):
    far = torch.zeros(66000, 65536, dtype=torch.bfloat16, device="cuda")
    far[65990:, :16] = 1
    y = h.dropout(far[:, :16], 0.5, key(41, 42), out=far[:, 16:32])
    want = kept(66000, 16, 0.5, 41, 42)[0].cuda()
    assert torch.equal(y[65990:] != 0, want[65990:]) and not y[:65990].any()


def test_empty(h):
    assert h.dropout(torch.empty(0, 8, device="cuda"), 0.5, key(1, 1)).shape == (0, 8)
    assert h.dropout(torch.empty(8, 0, device="cuda"), 0.5, key(1, 1)).shape == (8, 0)


def test_refusals(g, h):
    x, k = torch.zeros(4, 8, device="cuda"), key(1, 2)
    for p in (-0.1, 1.0, 0.999999, float("nan")):
        with pytest.raises(g.GemmError, match="INVALID_ARG"):
            h.dropout(x, p, k)
    with pytest.raises(TypeError):
        h.dropout(x, 0.5, k.int())
    with pytest.raises(ValueError):
        h.dropout(x, 0.5, k[:1])
    with pytest.raises(ValueError):
        h.dropout(x, 0.5, k.cpu())
    with pytest.raises(TypeError):
        h.dropout(x, 0.5, k, residual=x.half())
    with pytest.raises(TypeError):
        h.dropout(x, 0.5, k, out=x.half())
    with pytest.raises(TypeError):
        h.dropout(x.double(), 0.5, k)
    with pytest.raises(g.GemmError, match="INVALID_ARG"):
        h.dropout(x[:3], 0.5, k, out=x[1:])
