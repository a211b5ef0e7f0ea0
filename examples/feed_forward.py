"""A pre-norm gated feed-forward block on the library's operators,

    y = x + (silu(LN(x) Wg) * (LN(x) Wu)) Wd + bd,

with its backward pass, a plain gradient-descent step, and the single-token form that a
generation loop calls. ``python examples/feed_forward.py`` trains a small block to imitate
another one for some steps and then runs its tokens one at a time.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_tiled_gemm_05_gb300 as g  # noqa: E402


class FeedForward:
    """The block's parameters (weights as [outputs, inputs]) and its passes, on one handle."""

    def __init__(self, width, hidden, handle, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)

        def normal(rows, cols):
            w = torch.randn(rows, cols, generator=gen, device="cuda") * cols ** -0.5
            return w.to(dtype)

        self.h = handle
        self.w_gate, self.w_up = normal(hidden, width), normal(hidden, width)
        self.w_down = normal(width, hidden)
        self.b_down = torch.zeros(width, dtype=dtype, device="cuda")
        self.norm_w = torch.ones(width, device="cuda")
        self.norm_b = torch.zeros(width, device="cuda")

    def parameters(self):
        return [self.norm_w, self.norm_b, self.w_gate, self.w_up, self.w_down, self.b_down]

    def forward(self, x, out=None):
        """y for a batch of tokens (one or many rows); ``out=x`` adds onto the stream itself."""
        n = self.h.layer_norm(x, self.norm_w, self.norm_b)
        a = self.h.gated(n, self.w_gate.t(), self.w_up.t(), activation="silu")
        return self.h.matmul_epilogue(a, self.w_down.t(), bias=self.b_down, residual=x, out=out)

    def forward_saved(self, x):
        """y and what the backward pass reads."""
        n, mean, rstd = self.h.layer_norm(x, self.norm_w, self.norm_b, save=True)
        a, gate, up = self.h.gated(n, self.w_gate.t(), self.w_up.t(), activation="silu", save=True)
        y = self.h.matmul_epilogue(a, self.w_down.t(), bias=self.b_down, residual=x)
        return y, (x, n, mean, rstd, a, gate, up)

    def backward(self, dy, saved):
        """dx and the parameters' gradients, in the order of :meth:`parameters`."""
        x, n, mean, rstd, a, gate, up = saved
        da, dw_down, db_down = self.h.matmul_epilogue_backward(dy, a, self.w_down.t())
        dn, dw_gate, dw_up = self.h.gated_backward(da, n, self.w_gate.t(), self.w_up.t(), gate, up,
                                                   activation="silu")
        dx, dnw, dnb = self.h.layer_norm_backward(dn, x, self.norm_w, mean, rstd)
        dx += dy  # the residual's gradient
        return dx, [dnw, dnb, dw_gate.t(), dw_up.t(), dw_down.t(), db_down]


def train(block, teacher, steps, tokens, width, rate):
    """Gradient descent on the mean square distance of the two blocks' outputs."""
    gen = torch.Generator("cuda").manual_seed(9)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=gen, device="cuda").to(block.w_gate.dtype)
        y, saved = block.forward_saved(x)
        diff = y.float() - teacher.forward(x).float()
        losses.append(diff.square().mean())
        _, grads = block.backward((diff * (2.0 / tokens)).to(x.dtype), saved)
        for p, d in zip(block.parameters(), grads):
            p.sub_(d, alpha=rate)
    return [float(v) for v in losses]


def main(steps=60, tokens=512, width=256, hidden=1024):
    handle = g.Gemm(0)
    teacher = FeedForward(width, hidden, handle, seed=1)
    block = FeedForward(width, hidden, handle, seed=2)
    losses = train(block, teacher, steps, tokens, width, rate=0.05)
    x = torch.randn(tokens, width, device="cuda").to(torch.bfloat16)
    batch = block.forward(x)
    singles = torch.cat([block.forward(x[i:i + 1]) for i in range(32)])
    apart = float((singles.float() - batch[:32].float()).norm() / batch[:32].float().norm())
    status = handle.status()
    handle.close()
    print("loss %.4f -> %.4f over %d steps; 32 tokens one at a time differ from the batch by "
          "%.2g (status %d)" % (losses[0], losses[-1], steps, apart, status))
    return losses, apart, status


if __name__ == "__main__":
    main()
