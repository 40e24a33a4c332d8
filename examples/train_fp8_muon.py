"""Training with 8-bit products and Muon: a two-layer network fitted to a random teacher.

Every product of a linear layer runs through gemm_fp8: the forward x @ w.T (activations with a scale for each
1 x 128 group, weights for each 128 x 128 block), the input's gradient dy @ w (e5m2 against the turned weight) and the
weight's gradient dy.T @ x, contracted over the tokens and added to an fp32 gradient in place. quantize_fp8
hands out both orientations from one pass over its input. The update of each weight is its momentum
orthogonalised by newton_schulz.

    python examples/train_fp8_muon.py [--steps 30] [--width 1024] [--tokens 2048]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import thread_block_lds_amd as tbl  # noqa: E402


class Fp8Linear(torch.autograd.Function):
    """x (T, C) and an fp32 master weight w (N, C) -> x @ w.T in x's dtype; grad is the fp32 gradient of w that the
    backward adds to (w itself takes no part in autograd). The backward is not differentiable itself."""

    @staticmethod
    def forward(ctx, x, w, grad):
        xq, xt = tbl.quantize_fp8(x, transposed=True)
        wq, wt = tbl.quantize_fp8(w, rows=128, transposed=True)
        ctx.xt, ctx.wt, ctx.grad, ctx.dtype = xt, wt, grad, x.dtype
        return tbl.gemm_fp8(xq, wq, out_dtype=x.dtype)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        q, t = tbl.quantize_fp8(dy.contiguous(), fmt=torch.float8_e5m2, transposed=True)
        tbl.gemm_fp8(t, ctx.xt, add=ctx.grad, out=ctx.grad)
        return tbl.gemm_fp8(q, ctx.wt, out_dtype=ctx.dtype), None, None


class Muon:
    """Momentum whose matrix updates are orthogonalised."""

    def __init__(self, weights, lr, momentum=0.95):
        self.weights, self.lr, self.momentum = weights, lr, momentum
        self.buffers = [torch.zeros_like(w) for w in weights]

    def step(self, grads):
        for w, m, g in zip(self.weights, self.buffers, grads):
            m.mul_(self.momentum).add_(g)
            u = tbl.newton_schulz(g.add(m, alpha=self.momentum), out_dtype=torch.bfloat16)
            w.add_(u, alpha=-self.lr * max(1.0, w.shape[0] / w.shape[1]) ** 0.5)
            g.zero_()


def train(steps=30, width=1024, tokens=2048, lr=0.02, seed=0):
    """Returns the losses."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def weight(n, c):
        return torch.randn(n, c, generator=g, device="cuda") / c ** 0.5

    teacher = [weight(2 * width, width), weight(width, 2 * width)]
    weights = [weight(2 * width, width), weight(width, 2 * width)]
    grads = [torch.zeros_like(w) for w in weights]
    muon = Muon(weights, lr)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, generator=g, device="cuda")
        with torch.no_grad():
            want = torch.relu(x @ teacher[0].t()) @ teacher[1].t()
        h = Fp8Linear.apply(x.bfloat16().requires_grad_(), weights[0], grads[0])
        y = Fp8Linear.apply(torch.relu(h), weights[1], grads[1])
        loss = (y.float() - want).square().mean()
        loss.backward()
        muon.step(grads)
        losses.append(loss.item())
    return losses


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--steps", type=int, default=30)
    p.add_argument("--width", type=int, default=1024)
    p.add_argument("--tokens", type=int, default=2048)
    a = p.parse_args()
    for i, v in enumerate(train(a.steps, a.width, a.tokens)):
        print(f"step {i:3d}  loss {v:.4f}", flush=True)
