"""Layer norm on the GPU against plain 64-bit formulas.

Tolerances are rounding counts: an output rounded to a type t is off by at most
half a step, H[t] = finfo(t).eps / 2 of its magnitude; a float32 sum over a row
by at most A U of the sum of magnitudes, U = 2^-24, A = 90: 32 terms in a lane,
6 additions across a wave, 16 across waves, the division, and slack for terms
that were rounded themselves."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

from test_gpu_linear import BF, F32, H, HF, NORM_SHAPES, TINY, U, check_eight, randn, shifted, strided, within  # noqa: E402

A = 90
# rows of less than eight columns, one column past what a kernel holds, several rounds of rows in every kernel
MORE_SHAPES = [(5, 3), (9, 7), (600, 6), (70, 9), (3, 1537), (3, 2049), (2, 6145), (2, 12289), (2600, 513), (2100, 1032),
               (2100, 1300), (2100, 1800), (1100, 2304), (600, 4500), (600, 7000), (530, 8200), (530, 13000)]


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


def reference(h, w, b, eps):
    """(mean, its tolerance, rstd, its, y, the float32 y's) from the stored h."""
    h = h.double()
    mean = h.mean(1, keepdim=True)
    c = h - mean
    var = c.square().mean(1, keepdim=True)
    rstd = (var + eps) ** -0.5
    y = c * rstd * w.double() + (0.0 if b is None else b.double())
    # the first mean is off by `first`; what is left of the mean after the second look, by e_tol
    first = A * U * h.abs().mean(1, keepdim=True)
    d = c.abs().mean(1, keepdim=True) + first
    e_tol = A * U * d
    var_tol = A * U * (var + first.square()) + 2 * first * e_tol + e_tol.square()
    r_tol = rstd * (0.5 * var_tol / (var + eps) + 6 * U)
    y_tol = w.double().abs() * (rstd * (2 * U * (c.abs() + first) + e_tol) + r_tol * (c.abs() + e_tol)) + 4 * U * (y.abs() + (c * rstd * w.double()).abs())
    return mean[:, 0], (mean.abs() * U + e_tol)[:, 0], rstd[:, 0], r_tol[:, 0], y, y_tol


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("rows, width", NORM_SHAPES + MORE_SHAPES)
def test_forward(dev, rows, width, t):
    x = (randn(dev, 1, rows, width).mul_(3) + 2 * randn(dev, 11, rows, 1)).to(t)
    r = randn(dev, 2, rows, width).to(t)
    w, b = 1 + 0.2 * randn(dev, 3, width), 0.3 * randn(dev, 4, width)
    for eight, res, w_, b_ in (("e4m3", r, w, b), ("e5m2", None, w.to(t), b.to(t)), (None, r, w.to(t), None)):
        out = mr.layer_norm_forward(x, w_, b_, 1e-5, residual=res, eight=eight)
        if res is None:
            assert out.h is x
        else:
            want = x.double() + r.double()
            within(out.h, want, want.abs() * (H[t] + U) + TINY[t], "h")
        mean, m_tol, rstd, r_tol, y, y_tol = reference(out.h, w_, b_, 1e-5)
        within(out.mean, mean, m_tol + TINY[F32], "mean")
        within(out.rstd, rstd, r_tol, "rstd")
        within(out.y, y, y.abs() * H[t] * 1.01 + y_tol + TINY[t], "y")
        if eight:
            check_eight(out.q, out.scales, y, eight, False, y_tol)
        else:
            assert out.q is None and out.scales is None


@pytest.mark.parametrize("width", [1, 7, 100, 1000, 2048, 5000])
def test_rows_far_from_zero(dev, width):
    """Rows of equal values give the bias, rows of a small spread around a large value their norm."""
    w, b = 1 + 0.2 * randn(dev, 3, width), 0.3 * randn(dev, 4, width)
    c = torch.tensor([0.1, 1000.3, -77777.7, 3e8, 0.0], device=dev)
    x = c[:, None].expand(-1, width).contiguous()
    out = mr.layer_norm_forward(x, w, b, 1e-5)
    # the first mean is off by A U |c| at most, the second look leaves A U of that
    tol = (A * U) ** 2 * c.double().abs()[:, None] / 1e-5 ** 0.5 * w.double().abs() + 2 * U * b.double().abs()
    within(out.y, b.double().expand(5, -1), tol)
    within(out.mean, c.double(), c.double().abs() * 2 * U)
    x = (1000 + randn(dev, 5, 40, width))
    mean, m_tol, rstd, r_tol, y, y_tol = reference(x, w, b, 1e-5)
    out = mr.layer_norm_forward(x, w, b, 1e-5)
    within(out.mean, mean, m_tol)
    within(out.rstd, rstd, r_tol)
    within(out.y, y, y_tol + U * y.abs())


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows, width", [(5, 1024), (3, 333), (4, 4096)])
def test_strides_and_alignment(dev, rows, width, t):
    x, r, dy = (randn(dev, s, rows, width).to(t) for s in (4, 5, 7))
    w, b = 1 + 0.2 * randn(dev, 6, width), randn(dev, 8, width)
    want = mr.layer_norm_forward(x, w, b, 1e-6, residual=r, eight="e4m3")
    back = mr.layer_norm_backward(dy, want.h, want.mean, want.rstd, w, dresidual=r)
    for lay in (lambda v: strided(v, width + 24), lambda v: strided(v, width + 3), shifted):
        got = mr.layer_norm_forward(lay(x), w, b, 1e-6, residual=lay(r), eight="e4m3")
        for g, e in zip(got, want):
            assert torch.equal(g.float(), e.float())
        got = mr.layer_norm_backward(lay(dy), lay(want.h), want.mean, want.rstd, w, dresidual=lay(r))
        for g, e in zip(got, back):
            assert torch.equal(g, e)


def grad_reference(dy, h, mean, rstd, w, dres):
    """(dx, float32 tolerance, dweight, its, dbias, its)"""
    dy, h, w = dy.double(), h.double(), w.double()
    rows, width = dy.shape
    rho = rstd.double()[:, None]
    hh = (h - mean.double()[:, None]) * rho
    g = dy * w
    c0, c1 = g.mean(1, keepdim=True), (g * hh).mean(1, keepdim=True)
    dx = rho * (g - c0 - hh * c1) + (0.0 if dres is None else dres.double())
    tol = rho * (A * U * (g.abs().mean(1, keepdim=True) + hh.abs() * (g * hh).abs().mean(1, keepdim=True))
                 + 8 * U * (g.abs() + c0.abs() + (hh * c1).abs())) + 2 * U * dx.abs()
    # a column: the workgroup's rows one after another, its waves, the workgroups by 32 lanes and those
    n = rows / 512 + 1 + 4 + 16 + 32 + 4
    return dx, tol, (dy * hh).sum(0), n * U * (dy * hh).abs().sum(0), dy.sum(0), n * U * dy.abs().sum(0)


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("rows, width", NORM_SHAPES + MORE_SHAPES)
def test_backward(dev, rows, width, t):
    h, dy, dres = (randn(dev, s, rows, width).to(t) for s in (1, 2, 3))
    h = (h.float() * 2 + 1).to(t)
    w = 1 + 0.2 * randn(dev, 4, width)
    mean, _, rstd, _, _, _ = reference(h, w, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    for w_, r in ((w, dres), (w.to(t), None)):
        dx, x_tol, dw, w_tol, db, b_tol = grad_reference(dy, h, mean, rstd, w_, r)
        got = mr.layer_norm_backward(dy, h, mean, rstd, w_, dresidual=r)
        within(got[0], dx, dx.abs() * H[t] * 1.01 + x_tol + TINY[t], "dx")
        within(got[1], dw, w_tol, "dweight")
        within(got[2], db, b_tol, "dbias")
    dx, dw, db = mr.layer_norm_backward(dy, h, mean, rstd, w, weight_grad=False)
    assert dw is None and db is None
    assert torch.equal(dx, mr.layer_norm_backward(dy, h, mean, rstd, w)[0])


def test_gradients_against_differences(dev):
    """The loss sum(c y) of the kernel's float32 forward pass by differences of the 64-bit formula."""
    rows, width = 3, 37
    x, c, w, b = randn(dev, 1, rows, width), randn(dev, 2, rows, width), 1 + 0.2 * randn(dev, 3, width), randn(dev, 4, width)
    out = mr.layer_norm_forward(x, w, b, 1e-3)
    dx, dw, db = mr.layer_norm_backward(c, out.h, out.mean, out.rstd, w)

    def loss(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return (c.double() * (d * (d.square().mean(1, keepdim=True) + 1e-3) ** -0.5 * w + b)).sum()

    at = [v.double() for v in (x, w, b)]
    s = 1e-5
    for k, got in ((0, dx), (1, dw), (2, db)):
        for i in range(0, at[k].numel(), 5):
            step = torch.zeros_like(at[k])
            step.view(-1)[i] = s
            up, down = [v.clone() for v in at], [v.clone() for v in at]
            up[k], down[k] = at[k] + step, at[k] - step
            want = float(loss(*up) - loss(*down)) / (2 * s)
            # third derivatives times s^2 / 6 and 64-bit rounding over s are below 1e-7, the kernel's sums below 100 U of them
            assert abs(float(got.view(-1)[i]) - want) < 1e-6 + 1e-5 * max(1.0, abs(want)), (k, i)


def test_values_that_are_no_numbers_stay_in_their_rows(dev):
    rows, width = 9, 500
    w, b = torch.ones(width, device=dev), torch.zeros(width, device=dev)
    x = randn(dev, 1, rows, width)
    want = mr.layer_norm_forward(x, w, b, 1e-5, eight="e4m3")
    x[2, 499], x[5, 0], x[7, 3] = float("nan"), float("inf"), float("-inf")
    got = mr.layer_norm_forward(x, w, b, 1e-5, eight="e4m3")
    bad = torch.zeros(rows, dtype=torch.bool, device=dev)
    bad[[2, 5, 7]] = True
    for g, e in zip(got[1:], want[1:]):
        assert torch.equal(g[~bad].float(), e[~bad].float())
    assert bool(got.y[bad].isnan().all()) and bool(got.scales[bad].isnan().all())


def test_no_rows(dev):
    w = torch.ones(40, device=dev)
    x = torch.empty(0, 40, dtype=BF, device=dev)
    out = mr.layer_norm_forward(x, w, w, 1e-5, residual=x, eight="e4m3")
    assert out.y.shape == (0, 40) and out.mean.shape == (0,)
    dx, dw, db = mr.layer_norm_backward(x, x, out.mean, out.rstd, w)
    assert dx.shape == (0, 40) and bool((dw == 0).all()) and bool((db == 0).all())


def test_rows_past_four_gigabytes(dev):
    rows, width = 300000, 8192  # 4.9e9 bytes of bf16
    x = torch.zeros(rows, width, dtype=BF, device=dev)
    x[-3:] = randn(dev, 1, 3, width).to(BF)
    w, b = 1 + 0.2 * randn(dev, 3, width), randn(dev, 4, width)
    y = mr.layer_norm_forward(x, w, b, 1e-5).y
    want = mr.layer_norm_forward(x[-3:].clone(), w, b, 1e-5).y
    assert torch.equal(y[-3:], want) and torch.equal(y[1], b.to(BF))


def test_another_stream_and_a_captured_call(dev):
    x, dy = randn(dev, 1, 700, 640).to(BF), randn(dev, 2, 700, 640).to(BF)
    w, b = 1 + 0.2 * randn(dev, 3, 640), randn(dev, 4, 640)

    def both(**k):
        out = mr.layer_norm_forward(x, w, b, 1e-5, residual=dy, **k)
        return [*out[:4], *mr.layer_norm_backward(dy, out.h, out.mean, out.rstd, w, **k)]

    want = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = both(stream=s)
    s.synchronize()
    assert all(torch.equal(g, e) for g, e in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    for seed in range(3):
        x.copy_(randn(dev, 10 + seed, 700, 640))
        graph.replay()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(g, e) for g, e in zip(kept, want))
