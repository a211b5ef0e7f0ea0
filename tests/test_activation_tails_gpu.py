"""Activations and their slopes over -12 <= z <= 12 with relative bounds, so that the lower tails
count: products of one input z and a weight of 1 (exact in every kernel), fp32 outputs.

Bounds, relative to the sum of the magnitudes of the terms that a formula adds up: 3e-6 for the
approximations (exponential and reciprocal 2 ulps each, the normal tail's fit, a few roundings), and for the rounding of an exponent's argument t, formed in at most five steps,
5 2^-24 |t|: the relative error of e^t is the absolute one of t. Where a sigmoid s is close to 1,
s (1 - s) carries s's own rounding of 2^-24, times z and, for tanh-gelu, its inner slope w. What
is smaller than the least normal number may be flushed to 0, times up to 400 for z w."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ACTS = ["relu", "gelu", "gelu_tanh", "silu", "sigmoid"]
FLUSH = 400 * 2.0 ** -126
C = 2 * math.sqrt(2 / math.pi)  # tanh-gelu is z sigmoid(C (z + 0.044715 z^3))


def points():
    """Values of every size up to 12 (bf16 holds all, f16 those above its subnormals' spacing: the
    definitions take them as a type holds them)."""
    fine = torch.linspace(-12, 12, 4801).bfloat16()
    small = torch.tensor([s * 2.0 ** -k for k in range(1, 14) for s in (1, -1)]).bfloat16()
    return torch.unique(torch.cat([fine, small, torch.zeros(1).bfloat16()]).float()).cuda()


def definition(z, act):
    """(value, slope, |t|, magnitude of the slope's terms, rounding of s (1 - s)) in 64 bits."""
    z = z.double()
    if act == "relu":
        return z.clamp(min=0), (z > 0).double(), 0 * z, (z > 0).double(), 0 * z
    if act == "gelu":
        phi = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        p = 0.5 * torch.special.erfc(-z / math.sqrt(2))
        return z * p, p + z * phi, z * z / 2, p + z.abs() * phi, 0 * z
    if act == "gelu_tanh":
        t, w = C * (z + 0.044715 * z ** 3), C * (1 + 3 * 0.044715 * z * z)
    else:
        t, w = z, torch.ones_like(z)
    s, r = 1 / (1 + torch.exp(-t)), 1 / (1 + torch.exp(t))  # r = 1 - s
    near = 2.0 ** -23 * s * (z.abs() * w if act != "sigmoid" else 1) * (z > 0)
    if act == "sigmoid":
        return s, s * r, t.abs(), s * r, near
    return z * s, s + z * s * r * w, t.abs(), s + z.abs() * s * r * w, near


def assert_close(got, want, magnitude, t, extra=0.0):
    bound = (3e-6 + 5 * 2.0 ** -24 * t) * magnitude + extra + FLUSH
    over = (got.double() - want).abs() - bound
    i = int(over.argmax())
    assert float(over.max()) <= 0, "at point %d: %.9g, want %.9g, bound %.3g" % (
        i, float(got[i]), float(want[i]), float(bound[i]))


@pytest.fixture()
def h():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    import dense_tiled_gemm_05_gb300 as g
    hh = g.Gemm(0)
    yield hh
    assert hh.status() == 0
    hh.close()


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,cta_pair", [("bf16", 1), ("bf16", 2), ("f16", 1), ("f16", 2), ("f32", 0)])
@pytest.mark.parametrize("columns", [8, 5])
def test_values_by_rows(h, columns, dtype, cta_pair, act):
    """Tensor-core kernels, and the fp32 kernels: z down the rows."""
    z, t = points(), TYPES[dtype]
    a, b = z.to(t)[:, None], torch.ones(1, columns, dtype=t, device="cuda")
    h.set_option("cta_pair", cta_pair)
    want, _, arg, _, _ = definition(a[:, 0], act)
    for precision in ("default",) if dtype != "f32" else ("default", "tf32"):
        y = h.matmul_epilogue(a, b, activation=act, out_dtype="f32", precision=precision)
        for j in range(columns):
            assert_close(y[:, j], want, want.abs(), arg)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("tokens", [1, 4])
def test_values_by_features(h, tokens, dtype, act):
    """The kernel of few tokens: z over the features."""
    z, t = points(), TYPES[dtype]
    a, w = torch.ones(tokens, 1, dtype=t, device="cuda"), z.to(t)[:, None]
    want, _, arg, _, _ = definition(w[:, 0], act)
    y = h.matmul_epilogue(a, w.t(), activation=act, out_dtype="f32")
    for row in y:
        assert_close(row, want, want.abs(), arg)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("tokens", [1, 40])
def test_gated_values_in_32_bits(h, tokens, act):
    z = points()
    x, ones = torch.ones(tokens, 1, device="cuda"), torch.ones(1, len(z), device="cuda")
    want, _, arg, _, _ = definition(z, act)
    for row in h.gated(x, z[None, :], ones, activation=act):
        assert_close(row, want, want.abs(), arg)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("kept", list(TYPES))
@pytest.mark.parametrize("dtype", list(TYPES))
def test_slopes(h, dtype, kept, act):
    """One row of z and a gradient of 1: the bias gradient is the slope, in fp32."""
    z, t = points(), TYPES[dtype]
    n = len(z) // 8 * 8
    for z in (z[:n], z[:-1] if len(z) % 8 == 0 else z):  # with 16-byte accesses and without
        a, w = torch.ones(1, 4, dtype=t, device="cuda"), torch.ones(4, len(z), dtype=t, device="cuda")
        pre = z.to(TYPES[kept])[None, :]
        _, _, d = h.matmul_epilogue_backward(torch.ones_like(pre), a, w, pre=pre, activation=act,
                                             need=(False, False, True), bias_dtype="f32")
        _, want, arg, magnitude, near = definition(pre[0], act)
        assert_close(d, want, magnitude, arg, near)


@pytest.mark.parametrize("act", ACTS)
def test_gated_slopes_in_32_bits(h, act):
    """dx = dg + du of one feature with weights of 1 and 0: each of the two alone."""
    z = points()
    g, one = z[:, None].contiguous(), torch.ones(1, 1, device="cuda")
    value, slope, arg, magnitude, near = definition(z, act)
    dh, u, x = torch.ones_like(g), torch.ones_like(g), torch.ones_like(g)
    dx, _, _ = h.gated_backward(dh, x, one, 0 * one, g, u, activation=act)
    assert_close(dx[:, 0], slope, magnitude, arg, near)
    dx, _, _ = h.gated_backward(dh, x, 0 * one, one, g, u, activation=act)
    assert_close(dx[:, 0], value, value.abs(), arg)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,cta_pair,tokens", [("bf16", 1, 0), ("bf16", 2, 0), ("f16", 1, 0),
                                                   ("f16", 2, 0), ("f32", 0, 0), ("bf16", 0, 1),
                                                   ("f16", 0, 3), ("f32", 0, 1)])
@pytest.mark.parametrize("long", [False, True])
def test_fp32_outputs_have_fp32_activations(h, long, dtype, cta_pair, tokens, act):
    """Also from 16-bit operands: 4 ulps of the complementary error function, or 2 of the
    exponential, one of the reciprocal, 3e-7 of the tail's fit and two products, are below 1e-6.
    (long: zeros up to a K that the few-token kernel shares out over a cluster.)"""
    z, t = points(), TYPES[dtype]
    k = 2048 if long else 1
    x, w = torch.zeros(max(tokens, 1) if tokens else len(z), k, dtype=t, device="cuda"), None
    if tokens:
        w = torch.zeros(len(z), k, dtype=t, device="cuda")
        x[:, 0], w[:, 0] = 1, z.to(t)
        kept = w[:, 0]
    else:
        w = torch.zeros(8, k, dtype=t, device="cuda")
        x[:, 0], w[:, 0] = z.to(t), 1
        kept = x[:, 0]
    h.set_option("cta_pair", cta_pair)
    want, _, arg, _, _ = definition(kept, act)
    y = h.matmul_epilogue(x, w.t(), activation=act, out_dtype="f32")
    for v in y if tokens else y.t():
        over = (v.double() - want).abs() - (1e-6 + 5 * 2.0 ** -24 * arg) * want.abs() - FLUSH
        i = int(over.argmax())
        assert float(over.max()) <= 0, "at point %d: %.9g, want %.9g" % (i, float(v[i]), float(want[i]))
