"""A residual block of a model trained with the library's operators and steps.

    python -m matrix_roots_amd.layer_step [--steps K] [--tokens T]

The block is norm -> 8-bit linear layer -> one expert per token, added to its
input; it learns the outputs of a block with other weights:

    n = norm(x + r),  u = n W^T (8-bit operands),  z_t = V_e(t) u_t,  out = x + r + z

Its forward and backward pass are the linear-layer operators (linear.py), and
every weight matrix takes the optimizer's step on the float32 gradients they
give: Gram EMAs, their inverse quarter roots, the preconditioned direction, and
the norm-preserving hyperball update (binding.py).  All inputs are synthetic.
Prints the loss before every step.
"""

from __future__ import annotations

import argparse
from typing import List

import torch

from . import binding as B
from . import linear as L

EPS = 1e-6


class Block:
    """Weights of the block in float32 (width -> hidden -> width), and the products' forms of them."""

    def __init__(self, width: int, hidden: int, experts: int, seed: int, device):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.norm = torch.ones(width, device=device)
        self.w = torch.randn(hidden, width, generator=g, device=device) / width ** 0.5
        self.v = torch.randn(experts, width, hidden, generator=g, device=device) / hidden ** 0.5
        self.refresh()

    def refresh(self):
        """The operands of the products from the float32 weights: once per step."""
        self.w8 = L.quantize_blocks(self.w, "e4m3", block="square", order="both")
        self.v16 = self.v.bfloat16()

    def forward(self, x, residual, offsets):
        n = L.rms_norm_forward(x, self.norm, EPS, residual=residual, eight="e4m3")
        u = L.block_scaled_matmul(n.q, n.scales, self.w8.q, self.w8.scales)
        z = L.grouped_matmul(u, self.v16, offsets)
        return n.h + z, (n, u)

    def backward(self, dout, kept, offsets):
        """(dx, gradients of norm, w and v) from the gradient of the output."""
        n, u = kept
        du = L.grouped_matmul(dout, self.v16, offsets, transpose=True)
        dv = L.grouped_weight_grad(dout, u, offsets)
        d8 = L.quantize_blocks(du, "e5m2", order="both")
        dn = L.block_scaled_matmul(d8.q, d8.scales, self.w8.qt, self.w8.scales_t)
        n8 = L.quantize_blocks(n.y, "e4m3", order="columns")
        dw = L.block_scaled_matmul(d8.qt, d8.scales_t, n8.qt, n8.scales_t, out_dtype=torch.float32)
        dx, dnorm = L.rms_norm_backward(dn, n.h, n.rstd, self.norm, dresidual=dout)
        return dx, dnorm, dw, dv


class Optimizer:
    """Preconditioned hyperball steps of a list of float32 matrices."""

    def __init__(self, weights: List, beta: float = 0.9, eps: float = 1e-6, lr: float = 0.05):
        dev = weights[0].device
        self.weights, self.beta, self.eps, self.lr = weights, beta, eps, lr
        self.left = [torch.zeros(w.shape[0], w.shape[0], dtype=torch.float64, device=dev) for w in weights]
        self.right = [torch.zeros(w.shape[1], w.shape[1], dtype=torch.float64, device=dev) for w in weights]
        self.workspace = B.RootWorkspace()

    def step(self, grads: List):
        B.gram_ema_update(grads, self.left, self.right, self.beta)
        roots, _ = B.inv_quarter_root_batched(self.left + self.right, self.eps, workspace=self.workspace,
                                              return_info=False)
        n = len(grads)
        B.hyperball_update_batched(self.weights, B.precondition_apply(roots[:n], grads, roots[n:]), self.lr)


def train(steps: int = 10, tokens: int = 1000, width: int = 256, hidden: int = 384, experts: int = 6, seed: int = 0,
          log=None) -> List[float]:
    """The losses before each of `steps` steps and after the last one."""
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    x = torch.randn(tokens, width, generator=g, device=dev).bfloat16()
    residual = torch.randn(tokens, width, generator=g, device=dev).bfloat16()
    # tokens sorted by expert, uneven groups
    share = torch.rand(experts, generator=g, device=dev).cumsum(0)
    offsets = torch.cat([torch.zeros(1, device=dev), (share / share[-1] * tokens).round()]).to(torch.int32)
    target, _ = Block(width, hidden, experts, seed + 1, dev).forward(x, residual, offsets)
    block = Block(width, hidden, experts, seed + 2, dev)
    optimizer = Optimizer([block.w, *block.v.unbind(0)])
    losses = []
    for k in range(steps + 1):
        out, kept = block.forward(x, residual, offsets)
        gap = out.float() - target.float()
        losses.append(float(gap.square().mean()))
        if log is not None:
            log(f"step {k}: loss {losses[-1]:.4f}")
        if k == steps:
            return losses
        _, _, dw, dv = block.backward(gap.bfloat16(), kept, offsets)
        optimizer.step([dw, *dv.unbind(0)])
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
