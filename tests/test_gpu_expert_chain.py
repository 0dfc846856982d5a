"""The gradients of a block of experts on the GPU, from the values that its forward
pass stored, against the same chain in 64 bits (expert_chain.py)."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from matrix_roots_amd import binding as B  # noqa: E402
from matrix_roots_amd import expert_step as S  # noqa: E402

from expert_chain import bank_gradients, block_gradients, block_inputs, norm  # noqa: E402
from test_gpu_experts import block, chosen_of  # noqa: E402
from test_gpu_linear import BF, H, U, randn, within  # noqa: E402


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("tokens, width, experts, k", [(20, 64, 2, 1), (37, 128, 5, 2), (64, 256, 8, 3)])
def test_block(dev, tokens, width, experts, k):
    one = S.Block(width, experts, k, 3, dev)
    one.weight += 0.1 * randn(dev, 1, width)
    one.bias += 0.1 * randn(dev, 2, width)
    x, dout = block_inputs(tokens, width, 3, dev)
    out, kept = one.forward(x)
    n, logits, routed, order, rows, y = kept
    e = routed.experts.long()
    assert torch.equal(e, chosen_of(logits, k))
    assert torch.equal(rows[order.place.long()], n.y[:, None].expand(-1, k, -1))
    v, y_of = one.v16.double(), y[order.place.long()].double()
    want = (v[e] @ n.y.double()[:, None, :, None])[..., 0]
    size = (v[e].abs() @ n.y.double().abs()[:, None, :, None])[..., 0]
    within(y_of, want, want.abs() * H[BF] * 1.01 + 2 * width * U * size, "y")
    share = torch.softmax(logits.double().gather(1, e), 1)
    # k shares: their exps, the sum, the quotient, and differences of logits below 8
    within(routed.weights, share, share * (k + 30) * U, "weights")
    w = routed.weights.double()
    want = x.double() + (w[:, :, None] * y_of).sum(1)
    within(out, want, want.abs() * H[BF] * 1.01 + (k + 2) * U * (x.double().abs() + (w[:, :, None] * y_of.abs()).sum(1)), "out")
    got = dict(zip(("dx", "dweight", "dbias", "drouter", "dv"), one.backward(dout, kept)))
    for name, (g, tol) in block_gradients(dout, one.weight, one.router, one.v16, n.h, n.mean, n.rstd, n.y, e, w, y_of).items():
        assert got[name].shape == g.shape
        assert norm(got[name].double() - g) <= tol + 1e-30, (name, norm(got[name].double() - g), tol, norm(g))
        assert tol < 0.5 * norm(g) or (k == 1 and name == "drouter"), name


def test_run_of_operators(dev):
    """The bank's and the inputs' gradients of the run in test_gpu_experts.py, which adds no router's path."""
    tokens, width, n, k = 77, 128, 6, 2
    x, wr, bank = randn(dev, 1, tokens, width).to(BF), randn(dev, 2, width, n) / 16, (randn(dev, 3, n, width, width) / 11).to(BF)
    out, dbank, dx, _, weights, _ = block(x, wr, bank, k)
    e = chosen_of(x.float() @ wr, k)
    want = bank_gradients((out.float() * 0.01).to(BF), x, e, weights, bank)
    for got, name in ((dbank, "dv"), (dx, "dn")):
        g, tol = want[name]
        assert tol < 0.5 * norm(g)
        assert norm(got.double() - g) <= tol, name
