"""The linear-layer operators and the optimizer's step together, as a model
uses them (matrix_roots_amd.layer_step), and sizes that reach the operators'
largest and middle tiles, with ragged edges everywhere."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402
from matrix_roots_amd import layer_step  # noqa: E402

U = 2.0 ** -24
H = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


def randn(dev, seed, *shape):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=dev)


def test_the_block_learns(dev):
    """Every step moves each weight a fixed fraction of its norm along the preconditioned direction, so the loss
    falls step by step until that fraction is what is left."""
    losses = layer_step.train(steps=8, tokens=517)
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert losses[-1] < 0.5 * losses[0], losses
    assert layer_step.train(steps=2, tokens=517)[1:] == losses[1:3]  # the same bits again


def test_the_block_gradients_against_float64(dev):
    """dW, dV and dnorm of the block against the formula on the values that the 8-bit and 16-bit operands hold."""
    T, D, N, E = 300, 128, 256, 3
    block = layer_step.Block(D, N, E, 5, dev)
    x, r, dout = (randn(dev, s, T, D).bfloat16() for s in (1, 2, 3))
    off = torch.tensor([0, 100, 100, 300], dtype=torch.int32, device=dev)
    out, kept = block.forward(x, r, off)
    dx, dnorm, dw, dv = block.backward(dout, kept, off)
    n, u = kept
    h = n.h.double()
    rstd = (h.square().mean(1, keepdim=True) + layer_step.EPS) ** -0.5
    y = h * rstd
    w, v = block.w.double(), block.v16.double()
    e = torch.tensor([0] * 100 + [2] * 200, device=dev)
    du = torch.einsum("td,tdn->tn", dout.double(), v[e])
    want_dv = torch.zeros_like(v)
    for i in range(E):
        want_dv[i] = dout.double()[e == i].t() @ u.double()[e == i]
    within = lambda a, b, rel: float((a.double() - b).norm() / b.norm()) <= rel  # noqa: E731
    assert within(dv, want_dv, 1e-5)
    # operands in e4m3 (half step 2^-4) and e5m2 (2^-3): each value off by at most that
    assert within(dw, du.t().contiguous() @ y, 2.0 ** -4 + 2.0 ** -3)
    dn = du @ w
    assert within(dnorm, (dn * y).sum(0), 2 * (2.0 ** -4 + 2.0 ** -3))
    assert within(dx, dout.double() + rstd * (dn - y * (dn * y).mean(1, keepdim=True)), 2.0 ** -4 + 2.0 ** -3)


LARGE = [(8, 4000, 1104, 264), (8, 4000, 1100, 260), (3, 700, 520, 328), (64, 3000, 272, 264), (5, 900, 264, 1000)]


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("E, rows, n, k", LARGE)
def test_grouped_tiles(dev, E, rows, n, k, t):
    g = torch.Generator().manual_seed(E + rows)
    cut = torch.sort(torch.randint(0, rows - 20, (E - 1,), generator=g)).values.tolist()
    off = [7] + [max(7, c) for c in cut] + [rows - 9]
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    x, w, dy = randn(dev, 11, rows, k).to(t), randn(dev, 12, E, n, k).to(t), randn(dev, 13, rows, n).to(t)
    y, dx = mr.grouped_matmul(x, w, o, out_dtype=torch.float32), mr.grouped_matmul(dy, w, o, transpose=True)
    y16, dw = mr.grouped_matmul(x, w, o), mr.grouped_weight_grad(dy, x, o)
    assert torch.equal(y16, y.to(t))  # the same sums, rounded once
    for e in range(E):
        s = slice(off[e], off[e + 1])
        X, D, W = x[s].double(), dy[s].double(), w[e].double()
        for got, a, b, steps, h in ((y[s], X, W.t().contiguous(), k, U), (dx[s], D, W, n, H[t]),
                                    (dw[e], D.t().contiguous(), X, off[e + 1] - off[e], U)):
            want = a @ b
            tol = (a.abs() @ b.abs()) * 2 * (steps + 1) * U + want.abs() * h * 1.01 + 2.0 ** -24
            want, got = (want.clamp(-65504, 65504), got.clamp(-65504, 65504)) if t == torch.float16 else (want, got)
            assert bool(((got.double() - want).abs() <= tol).all()), (e, steps)
    assert bool((y[:7] == 0).all()) and bool((y[rows - 9:] == 0).all()) and bool((dx[:7] == 0).all())


def test_offsets_that_decrease_stay_inside(dev):
    """Not a valid grouping: nothing is promised but that the call ends and writes Y alone."""
    rows, n, k = 200, 96, 64
    x, w = randn(dev, 21, rows, k).bfloat16(), randn(dev, 22, 5, n, k).bfloat16()
    big = torch.full((rows + 64, n), 3.0, device=dev).bfloat16()
    for off in ([0, 150, 20, 200, 90, 200], [200, 100, 50, 0, 0, 0], [0, 200, 0, 200, 0, 200]):
        o = torch.tensor(off, dtype=torch.int64, device=dev)
        mr.grouped_matmul(x, w, o, out=big[32:32 + rows])
        mr.grouped_weight_grad(randn(dev, 23, rows, n).bfloat16(), x, o)
        torch.cuda.synchronize()
        assert bool((big[:32] == 3).all()) and bool((big[32 + rows:] == 3).all())


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("m", [5, 300])
def test_product_of_the_smallest_values(dev, m, out):
    """Subnormal e5m2 and e4m3 operands count in full: 2^-16 2^-9 summed 256 times is 2^-17, exactly."""
    a = torch.full((m, 256), 2.0 ** -16, device=dev).to(torch.float8_e5m2)
    b = torch.full((40, 256), 2.0 ** -9, device=dev).to(torch.float8_e4m3fn)
    c = mr.block_scaled_matmul(a, torch.ones(m, 2, device=dev), b, torch.ones(1, 2, device=dev), out_dtype=out)
    assert bool((c.double() == 2.0 ** -17).all())


@pytest.mark.parametrize("m", [5, 300, 4200])
def test_product_with_nothing_after_the_last_row(dev, m):
    """k no multiple of 16 and memory that ends with the last row (no padding to read), against the padded form."""
    n, k = 300 if m < 4000 else 4200, 136 + 7
    a, b = mr.quantize_blocks(randn(dev, 31, m, k)), mr.quantize_blocks(randn(dev, 32, n, k), block="square")
    tight = []
    for q in (a.q, b.q):
        rows, ld = q.shape[0], q.stride(0)
        flat = torch.zeros((rows - 1) * ld + k, dtype=q.dtype, device=dev)
        flat.as_strided((rows, k), (ld, 1)).copy_(q)
        tight.append(flat.as_strided((rows, k), (ld, 1)))
    want = mr.block_scaled_matmul(a.q, a.scales, b.q, b.scales)
    assert torch.equal(mr.block_scaled_matmul(tight[0], a.scales, tight[1], b.scales), want)
    # bytes of the padding are ignored, NaN (0x7f) among them
    pad = a.q.as_strided((m, a.q.stride(0)), a.q.stride())
    pad[:, k:].view(torch.uint8).fill_(0x7F)
    assert torch.equal(mr.block_scaled_matmul(a.q, a.scales, b.q, b.scales), want)


@pytest.mark.parametrize("m, n, k", [(3, 100, 9000), (16, 64, 16384), (40, 33, 8200), (200, 120, 12345)])
def test_product_split_over_a_long_contraction(dev, m, n, k):
    a = mr.quantize_blocks(randn(dev, 41, m, k))
    b = mr.quantize_blocks(randn(dev, 42, n, k), block="square")
    x = a.q.double() * a.scales.double().repeat_interleave(128, 1)[:, :k]
    w = b.q.double() * b.scales.double().repeat_interleave(128, 1)[:, :k].repeat_interleave(128, 0)[:n]
    want, mag = x @ w.t().contiguous(), x.abs() @ w.abs().t().contiguous()
    start = randn(dev, 43, m, n)
    c = start.clone()
    mr.block_scaled_matmul(a.q, a.scales, b.q, b.scales, out=c, accumulate=True)
    # 128 products of a block at 2 U, the blocks, 16 parts, the sum that was there
    tol = mag * (2 * 128 + (k + 127) // 128 + 3 + 16 + 2) * U + (want + start.double()).abs() * U * 1.01
    assert bool(((c.double() - (want + start.double())).abs() <= tol + 2.0 ** -24 * start.double().abs()).all())
    half = mr.block_scaled_matmul(a.q, a.scales, b.q, b.scales)
    assert bool(((half.double() - want).abs() <= mag * 2.0 ** -14 + want.abs() * 2.0 ** -8 * 1.01).all())
    assert torch.equal(half, mr.block_scaled_matmul(a.q, a.scales, b.q, b.scales))


def test_operators_are_traced(dev):
    B.trace_enable(True)
    try:
        layer_step.train(steps=1, tokens=64)
        seen = B.trace_collect()
    finally:
        B.trace_enable(False)
    for name in ("norm", "norm_grad", "quantize", "scaled_matmul", "grouped", "grouped_grad"):
        assert seen[name][0] > 0 and seen[name][1] > 0, name
