"""The 64-bit backward pass that the block of experts is checked against: it agrees
with autograd, its tolerances let bfloat16 rounding through and nothing that a
mistake in the chain would give."""

import pytest
import torch

from expert_chain import block_gradients, block_inputs, norm

SHAPES = [(37, 128, 5, 2), (64, 256, 8, 3)]
EPS = 1e-5


def forward(tokens, width, experts, k, seed=3):
    """The block's stored values, rounded where it rounds them."""
    g = torch.Generator().manual_seed(seed)
    x, dout = block_inputs(tokens, width, seed, "cpu")
    weight, bias = 1 + 0.1 * torch.randn(width, generator=g), 0.1 * torch.randn(width, generator=g)
    router = torch.randn(width, experts, generator=g) / width ** 0.5
    v = (torch.randn(experts, width, width, generator=g) / width ** 0.5).bfloat16()
    h = x.double()
    mean = h.mean(1)
    rstd = ((h - mean[:, None]).square().mean(1) + EPS) ** -0.5
    n = ((h - mean[:, None]) * rstd[:, None] * weight + bias).bfloat16()
    l = n.float() @ router
    top = torch.topk(l, k, dim=1)
    w = torch.softmax(top.values, 1)
    e = top.indices
    y = torch.stack([(v[e[:, j]].float() @ n.float()[:, :, None])[..., 0] for j in range(k)], 1).bfloat16()
    return dict(dout=dout, weight=weight, router=router, v=v, h=x, mean=mean.float(), rstd=rstd.float(), n=n, e=e, w=w, y=y)


def rounded(dout, weight, router, v, h, mean, rstd, n, e, w, y, wrong=""):
    """The block's backward pass as it is computed, bfloat16 and float32 where it has them; with a mistake."""
    (tokens, k), experts = e.shape, v.shape[0]
    dy = (w[:, :, None] * dout.float()[:, None]).bfloat16()
    if wrong == "no weights":
        dy = dout[:, None].expand(-1, k, -1)
    dv = torch.zeros(v.shape)
    for i in range(experts):
        t, j = torch.nonzero(e == i).unbind(1)
        dv[i] = dy[t, j].float().t() @ n[t].float()
    drows = torch.stack([(dy[:, j].float()[:, None] @ v[e[:, j]].float())[:, 0] for j in range(k)], 1).bfloat16()
    if wrong == "bank not transposed":
        drows = torch.stack([(v[e[:, j]].float() @ dy[:, j].float()[..., None])[..., 0] for j in range(k)], 1).bfloat16()
    dn = (drows[:, 0] if wrong == "one choice" else drows).float().view(tokens, -1, n.shape[1]).sum(1).bfloat16()
    dw = (y.float() * dout.float()[:, None]).sum(2)
    c = 0 if wrong == "no mean of weights" else (w * dw).sum(1, keepdim=True)
    dl = torch.zeros(tokens, experts).scatter_add_(1, e, w * (dw - c))
    drouter = n.float().t() @ dl
    if wrong != "no router":
        dn = (dn.float() + dl @ router.t()).bfloat16()
    hh = (h.float() - mean[:, None]) * rstd[:, None]
    g = dn.float() * weight
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - hh * (g * hh).mean(1, keepdim=True))
    if wrong == "no projection":
        dx = rstd[:, None] * g
    dx = (dx if wrong == "no residual" else dx + dout.float()).bfloat16()
    return {"dx": dx, "dweight": (dn.float() * hh).sum(0), "dbias": dn.float().sum(0), "drouter": drouter, "dv": dv}


def off(got, want):
    """{name: error over tolerance}"""
    return {name: norm(got[name].double() - g) / tol for name, (g, tol) in want.items()}


@pytest.mark.parametrize("shape", SHAPES)
def test_rounding_passes(shape):
    kept = forward(*shape)
    assert max(off(rounded(**kept), block_gradients(**kept)).values()) <= 1


@pytest.mark.parametrize("shape", SHAPES)
def test_the_chain_against_autograd(shape):
    """From the same stored values: the experts' outputs and the norm's are leaves of their own where they were rounded."""
    kept = forward(*shape)
    want = block_gradients(**kept)
    k, leaf = {a: t.double() if t.is_floating_point() else t for a, t in kept.items()}, {}
    for name in ("n", "v", "y", "router", "w"):
        leaf[name] = k[name].clone().requires_grad_()
    y = torch.stack([(leaf["v"][k["e"][:, j]] @ leaf["n"][:, :, None])[..., 0] for j in range(k["e"].shape[1])], 1)
    (dw,) = torch.autograd.grad((leaf["w"][:, :, None] * leaf["y"]).sum(1), leaf["w"], k["dout"])
    dn, dv = torch.autograd.grad((k["w"][:, :, None] * y).sum(1), [leaf["n"], leaf["v"]], k["dout"])
    # shares w of logits log w: the softmax's gradient at the stored weights
    l = torch.log(k["w"]).requires_grad_()
    (dl,) = torch.autograd.grad(torch.softmax(l, 1), l, dw * k["w"].sum(1, keepdim=True))
    logits = leaf["n"] @ leaf["router"]
    part, drouter = torch.autograd.grad(logits.gather(1, k["e"]), [leaf["n"], leaf["router"]], dl)
    h = k["h"].clone().requires_grad_()
    weight, bias = k["weight"].clone().requires_grad_(), torch.zeros_like(k["weight"]).requires_grad_()
    c = h - h.mean(1, keepdim=True)
    out = c * (c.square().mean(1, keepdim=True) + EPS) ** -0.5 * weight + bias
    dx, dweight, dbias = torch.autograd.grad(out, [h, weight, bias], dn + part)
    for name, g in (("dx", dx + k["dout"]), ("dweight", dweight), ("dbias", dbias), ("drouter", drouter), ("dv", dv)):
        # the stored float32 mean, rstd and weights (whose sum is not 1) are off by some 2^-24
        assert norm(want[name][0] - g) <= 1e-6 * (norm(g) + norm(dn)), name


@pytest.mark.parametrize("shape", SHAPES)
def test_mistakes_do_not_pass(shape):
    kept = forward(*shape)
    want = block_gradients(**kept)
    right = rounded(**kept)
    for name, (g, tol) in want.items():
        assert tol < 0.5 * norm(g), (name, tol / norm(g))  # neither zeros nor the negative pass
    assert want["dx"][1] < 0.5 * norm(want["dx"][0] - kept["dout"].double())  # nor the residual's path alone
    for wrong, names in (("no weights", ("dv", "dx", "dbias")), ("bank not transposed", ("dx", "dweight", "dbias")),
                         ("one choice", ("dx", "dbias")), ("no mean of weights", ("drouter",)), ("no router", ("dx", "dweight")),
                         ("no projection", ("dx",)), ("no residual", ("dx",))):
        got = off(rounded(**kept, wrong=wrong), want)
        assert all(got[n] > 1 for n in names), (wrong, got)
    assert all(v <= 1 for v in off(right, want).values())
