"""Plain 64-bit forms of the feed-forward operators and the bounds their kernels are held to.

Bounds, element by element (u: half a spacing of the stored type, D: the sum of the
magnitudes a sum adds up):

* a product of 16-bit operands is a sum of exact products in the tensor cores' fp32
  accumulator, which may drop up to 2^-22 of the running magnitude at each of its K / 16
  steps: (K / 16 + 8) 2^-22 D;
* exact fp32 products stay within 1e-6 D, tf32 ones within 2e-3 D;
* activations have slopes below 1.2 and are evaluated to 2^-20 (|z| + 1); their slopes are
  evaluated to 2^-19 (the second derivatives stay below 1.2);
* sums over n values a thread and a tree of at most 16 levels: (n + 16) 2^-24 D.
"""
import math

import torch

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
# half the spacing of the type's subnormals: the absolute floor of a rounding
TINY = {torch.float32: 2.0 ** -150, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"]


def act64(z, name):
    if name in (None, "none"):
        return z
    if name == "relu":
        return z.clamp(min=0)
    if name == "gelu":
        return z * torch.special.ndtr(z)
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    s = 1 / (1 + torch.exp(-z))
    return z * s if name == "silu" else s


def slope64(z, name):
    """act'(z) by automatic differentiation of the definition (relu: 0 at 0)."""
    if name in (None, "none"):
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    with torch.enable_grad():
        z = z.detach().clone().requires_grad_(True)
        return torch.autograd.grad(act64(z, name).sum(), z)[0]


def acc_error(dtype, K, precision="default"):
    """Relative bound (of D) on a K-long product's accumulation."""
    if dtype == torch.float32:
        return 2e-3 if precision == "tf32" else 1e-6
    return (K / 16 + 8) * 2.0 ** -22


def rounding(y, dtype):
    return UNIT[dtype] * y.abs() + TINY[dtype]


def assert_within(got, want, bound, what=""):
    got = got.double()
    assert got.shape == want.shape, what
    assert torch.isfinite(got).all(), "%s: not finite" % what
    if not got.numel():
        return
    over = (got - want).abs() - bound
    worst = int(over.argmax())
    assert float(over.max()) <= 0, "%s: off by %.3g, bound %.3g, at %d of %s (want %.6g)" % (
        what, float((got - want).abs().flatten()[worst]), float(
            torch.broadcast_to(bound, want.shape).flatten()[worst]), worst, tuple(want.shape),
        float(want.flatten()[worst]))


def matrix(rows, cols, dtype, seed, layout="row", pad=0, offset=0, scale=1.0, device="cuda"):
    """A rows x cols view of normal values; `pad` poisoned (NaN) elements after every line,
    `offset` elements before the first one."""
    gen = torch.Generator(device=device).manual_seed(seed)
    r, c = (rows, cols) if layout == "row" else (cols, rows)
    store = torch.full((offset + r * (c + pad),), float("nan"), dtype=dtype, device=device)
    view = store[offset:].view(r, c + pad)[:, :c]
    view.copy_((torch.randn(r, c, generator=gen, device=device) * scale).to(dtype))
    return view if layout == "row" else view.t()
