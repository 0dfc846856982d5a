"""The block of experts that expert_step.py trains: it runs, and its gradients are
those of its formula.

A gradient is compared with the 64-bit one (torch.autograd over the formula, with
the experts that the block chose).  Six values on the way are rounded to bf16 (the
norm's output, the experts' outputs, the output's gradient, the rows' two and the
norm's), and the weights once: eight times half a step of the same formula with
every term's magnitude."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from matrix_roots_amd import binding as B  # noqa: E402
from matrix_roots_amd import expert_step as S  # noqa: E402

from test_gpu_linear import BF, H, randn, within  # noqa: E402


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("tokens, width, experts, k", [(1, 64, 2, 1), (37, 128, 5, 2), (300, 256, 8, 3)])
def test_gradients(dev, tokens, width, experts, k):
    block = S.Block(width, experts, k, 3, dev)
    block.weight += 0.1 * randn(dev, 1, width)
    block.bias += 0.1 * randn(dev, 2, width)
    x, dout = randn(dev, 4, tokens, width).to(BF), (randn(dev, 5, tokens, width) / tokens).to(BF)
    out, kept = block.forward(x)
    got = block.backward(dout, kept)
    e = kept[2].experts.long()
    leaves = [v.double().requires_grad_() for v in (x, block.weight, block.bias, block.router, block.v16)]
    xd, w, b, r, v = leaves
    c = xd - xd.mean(1, keepdim=True)
    rho = (c.square().mean(1, keepdim=True) + S.EPS) ** -0.5
    hh = c * rho
    n = hh * w + b
    share = torch.softmax((n @ r).gather(1, e), 1)
    y = (v[e] @ n[:, None, :, None])[..., 0]
    want_out = xd + (share[:, :, None] * y).sum(1)
    want_out.backward(dout.double())
    with torch.no_grad():
        n_abs, d_abs = (hh * w).abs() + b.abs(), dout.double().abs()
        y_abs = (v.abs()[e] @ n_abs[:, None, :, None])[..., 0]
        # a weight is off by what its logits are: n's half steps through the router
        slack = 1 + 2 * (n_abs @ r.abs()).amax(1)
        out_abs = xd.abs() + slack[:, None] * (share[:, :, None] * y_abs).sum(1)
        within(out, want_out, 8 * H[BF] * out_abs, "out")
        dw_abs = (d_abs[:, None] * y_abs).sum(2)
        dl_abs = torch.zeros(tokens, experts, dtype=torch.float64, device=dev)
        dl_abs.scatter_add_(1, e, share * (dw_abs + (share * dw_abs).sum(1, keepdim=True)) * slack[:, None])
        dy_abs = slack[:, None, None] * share[:, :, None] * d_abs[:, None]
        dv_abs = torch.zeros_like(v)
        for t in range(tokens):
            for j in range(k):
                dv_abs[e[t, j]] += dy_abs[t, j][:, None] * n_abs[t][None]
        dn_abs = (v.abs().transpose(1, 2).contiguous()[e] @ dy_abs[..., None])[..., 0].sum(1) + dl_abs @ r.abs().t().contiguous()
        g_abs = dn_abs * w.abs()
        dx_abs = d_abs + rho * (g_abs + g_abs.mean(1, keepdim=True) + hh.abs() * (g_abs * hh.abs()).mean(1, keepdim=True))
        sizes = (dx_abs, (dn_abs * hh.abs()).sum(0), dn_abs.sum(0), n_abs.t().contiguous() @ dl_abs, dv_abs)
    for name, g, leaf, size in zip(("dx", "dweight", "dbias", "drouter", "dv"), got, leaves, sizes):
        within(g, leaf.grad, 8 * H[BF] * size + 1e-30, name)


def test_it_runs(dev):
    losses = S.train(steps=3, tokens=200, width=64, experts=4, log=lambda s: None)
    assert len(losses) == 4 and all(math.isfinite(v) for v in losses)
    assert S.main(["--steps", "1", "--tokens", "64"]) == 0
