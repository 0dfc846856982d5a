"""A residual block of experts trained with the library's operators and steps.

    python -m matrix_roots_amd.expert_step [--steps K] [--tokens T]

The block normalises its input, sends each token to its k best experts and adds
what they make of it, by the router's weights, to its input; it learns the
outputs of a block with other weights:

    n = layer_norm(x),  l = n R,  out_t = x_t + sum_j w_tj V_e(t,j) n_t

Forward and backward pass are the operators of linear.py and experts.py; the
gradients, clipped by their common norm, go to the optimizer's step (Gram EMAs,
inverse quarter roots, preconditioned direction, hyperball update), those of the
norm's vectors to a plain step.  All inputs are synthetic.  Prints the loss and
the gradients' norm before every step.
"""

from __future__ import annotations

import argparse
from typing import List

import torch

from . import binding as B
from . import experts as X
from . import linear as L
from .layer_step import Optimizer

EPS = 1e-5


class Block:
    """Weights of the block in float32, and the products' form of the experts'."""

    def __init__(self, width: int, experts: int, k: int, seed: int, device):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.k = k
        self.weight = torch.ones(width, device=device)
        self.bias = torch.zeros(width, device=device)
        self.router = torch.randn(width, experts, generator=g, device=device) / width ** 0.5
        self.v = torch.randn(experts, width, width, generator=g, device=device) / width ** 0.5
        self.refresh()

    def refresh(self):
        """The operand of the products from the float32 weights: once per step."""
        self.v16 = self.v.bfloat16()

    def forward(self, x):
        n = L.layer_norm_forward(x, self.weight, self.bias, EPS)
        logits = n.y.float() @ self.router
        routed = X.route_tokens(logits, self.k)
        order = X.order_by_expert(routed.experts, self.v.shape[0])
        rows = X.dispatch_rows(n.y, order)
        y = L.grouped_matmul(rows, self.v16, order.offsets)
        out = X.combine_rows(y, order, weights=routed.weights, residual=x)
        return out, (n, logits, routed, order, rows, y)

    def backward(self, dout, kept):
        """(dx, gradients of weight, bias, router and v) from the gradient of the output."""
        n, logits, routed, order, rows, y = kept
        dy, dw = X.combine_rows_backward(dout, y, order, routed.weights)
        dv = L.grouped_weight_grad(dy, rows, order.offsets)
        drows = L.grouped_matmul(dy, self.v16, order.offsets, transpose=True)
        dlogits = X.route_tokens_backward(dw, logits, routed)
        drouter = n.y.float().t() @ dlogits
        dn = (X.dispatch_rows_backward(drows, order).float() + dlogits @ self.router.t()).to(dout.dtype)
        dx, dweight, dbias = L.layer_norm_backward(dn, n.h, n.mean, n.rstd, self.weight, dresidual=dout)
        return dx, dweight, dbias, drouter, dv


def train(steps: int = 10, tokens: int = 1000, width: int = 256, experts: int = 6, k: int = 2, max_norm: float = 0.1,
          seed: int = 0, log=None) -> List[float]:
    """The losses before each of `steps` steps and after the last one."""
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.randn(tokens, width, generator=g, device=dev).bfloat16()
    target, _ = Block(width, experts, k, seed + 1, dev).forward(x)
    block = Block(width, experts, k, seed + 2, dev)
    optimizer = Optimizer([block.router, *block.v.unbind(0)])
    losses = []
    for step in range(steps + 1):
        out, kept = block.forward(x)
        gap = out.float() - target.float()
        losses.append(float(gap.square().mean()))
        if step == steps:
            if log is not None:
                log(f"step {step}: loss {losses[-1]:.4f}")
            return losses
        _, dweight, dbias, drouter, dv = block.backward((gap * (2 / gap.numel())).bfloat16(), kept)
        norm = B.clip_gradients_batched([dweight, dbias, drouter, dv], max_norm)
        if log is not None:
            log(f"step {step}: loss {losses[-1]:.4f}, gradients' norm {float(norm):.3g}")
        optimizer.step([drouter, *dv.unbind(0)])
        block.weight -= 0.01 * dweight
        block.bias -= 0.01 * dbias
        block.refresh()


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=10)
    ap.add_argument("--tokens", type=int, default=1000)
    a = ap.parse_args(argv)
    train(a.steps, a.tokens, log=print)
    return 0


if __name__ == "__main__":
    raise SystemExit(main())
