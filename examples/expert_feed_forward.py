"""A pre-norm feed-forward block split over experts, on the library's operators:

    n = LN(x),  the router's k largest logits of n Wr choose the experts, w = their softmax,
    y = x + dropout(sum_j w_j E_j(n)),   E_e(v) = (silu(v Wg_e) * (v Wu_e)) Wd_e,

with its backward pass, a plain gradient-descent step, and the form without dropout that a
generation loop calls for a few tokens. No count of rows goes to the host, so that a step can be
captured in a CUDA graph. ``python examples/expert_feed_forward.py`` trains a small block to imitate
another one for some steps and then runs some of its tokens one at a time.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_tiled_gemm_05_gb300 as g  # noqa: E402


class ExpertFeedForward:
    """The block's parameters (weights as [experts, outputs, inputs]) and its passes, on one handle."""

    def __init__(self, width, hidden, experts, choices, handle, drop=0.0, dtype=torch.bfloat16, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)

        def normal(*shape):
            return (torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5).to(dtype)

        self.h, self.experts, self.choices, self.drop = handle, experts, choices, drop
        self.router = normal(experts, width)
        self.w_gate, self.w_up = normal(experts, hidden, width), normal(experts, hidden, width)
        self.w_down = normal(experts, width, hidden)
        self.norm_w = torch.ones(width, device="cuda")
        self.norm_b = torch.zeros(width, device="cuda")
        # seed, and the number of the training step, on the device for captured steps
        self.key = torch.tensor([seed, 0], device="cuda")

    def parameters(self):
        return [self.norm_w, self.norm_b, self.router, self.w_gate, self.w_up, self.w_down]

    def route(self, n):
        """The tokens' experts and their weights (f32)."""
        logits = self.h.matmul(n, self.router.t(), out_dtype="f32")
        top, ids = logits.topk(self.choices, 1)
        return ids, self.h.softmax_rows(top)

    def forward(self, x, out=None):
        """y without dropout, for a few tokens or many; ``out=x`` adds onto the stream itself."""
        n = self.h.layer_norm(x, self.norm_w, self.norm_b)
        ids, weights = self.route(n)
        position, offsets = self.h.expert_sort(ids, self.experts)
        rows = self.h.expert_gather(n, position)
        a = self.h.expert_gated(rows, self.w_gate.transpose(1, 2), self.w_up.transpose(1, 2), offsets)
        z = self.h.expert_matmul(a, self.w_down.transpose(1, 2), offsets)
        return self.h.expert_combine(z, position, weights, residual=x, out=out)

    def forward_saved(self, x):
        """y of a training step and what the backward pass reads."""
        h = self.h
        n, mean, rstd = h.layer_norm(x, self.norm_w, self.norm_b, save=True)
        ids, weights = self.route(n)
        position, offsets = h.expert_sort(ids, self.experts)
        rows = h.expert_gather(n, position)
        a, gate, up = h.expert_gated(rows, self.w_gate.transpose(1, 2), self.w_up.transpose(1, 2), offsets,
                                     save=True)
        z = h.expert_matmul(a, self.w_down.transpose(1, 2), offsets)
        y = h.dropout(h.expert_combine(z, position, weights), self.drop, self.key, residual=x)
        return y, (x, n, mean, rstd, ids, weights, position, offsets, rows, a, gate, up, z)

    def backward(self, dy, saved):
        """dx and the parameters' gradients, in the order of :meth:`parameters`."""
        x, n, mean, rstd, ids, weights, position, offsets, rows, a, gate, up, z = saved
        h = self.h
        dc = h.dropout_backward(dy, self.drop, self.key)
        dz, dweights = h.expert_combine_backward(dc, z, position, weights)
        da, dw_down = h.expert_matmul_backward(dz, a, self.w_down.transpose(1, 2), offsets)
        drows, dw_gate, dw_up = h.expert_gated_backward(
            da, rows, self.w_gate.transpose(1, 2), self.w_up.transpose(1, 2), gate, up, offsets)
        dn = h.expert_gather_backward(drows, position)
        # the softmax of the chosen logits, and the router's product
        dtop = weights * (dweights - (weights * dweights).sum(1, keepdim=True))
        dlogits = torch.zeros(x.shape[0], self.experts, device="cuda").scatter_(1, ids, dtop).to(n.dtype)
        dn_router, d_router, _ = h.matmul_epilogue_backward(dlogits, n, self.router.t(),
                                                            need=(True, True, False))
        dn += dn_router
        dx, dnw, dnb = h.layer_norm_backward(dn, x, self.norm_w, mean, rstd)
        dx += dy  # the residual's gradient
        return dx, [dnw, dnb, d_router.t(), dw_gate.transpose(1, 2), dw_up.transpose(1, 2),
                    dw_down.transpose(1, 2)]


    def reference(self, x, dy, ids):
        """y, dx and the parameters' gradients of a training step in 64 bits, for these choices, by
        automatic differentiation (the mask is the library's, of ones)."""
        f = torch.nn.functional
        x = x.double().requires_grad_(True)
        nw, nb, wr, wg, wu, wd = ps = [p.double().requires_grad_(True) for p in self.parameters()]
        mask = self.h.dropout(torch.ones(x.shape, device="cuda"), self.drop, self.key).double()
        n = f.layer_norm(x, x.shape[1:], nw, nb)
        weights = (n @ wr.t()).gather(1, ids).softmax(1)
        y = x
        for e in range(self.experts):
            out = (f.silu(n @ wg[e].t()) * (n @ wu[e].t())) @ wd[e].t()
            y = y + mask * (weights * (ids == e)).sum(1, keepdim=True) * out
        return [y.detach()] + list(torch.autograd.grad(y, [x] + ps, dy.double()))


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
        block.key[1] += 1
        for p, d in zip(block.parameters(), grads):
            p.sub_(d, alpha=rate)
    return [float(v) for v in losses]


def main(steps=40, tokens=512, width=256, hidden=384, experts=8, choices=2):
    handle = g.Gemm(0)
    teacher = ExpertFeedForward(width, hidden, experts, choices, handle, seed=1)
    block = ExpertFeedForward(width, hidden, experts, choices, handle, drop=0.05, seed=2)
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
