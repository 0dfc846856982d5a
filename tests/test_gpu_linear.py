"""The linear-layer operators on the GPU against plain 64-bit formulas.

Tolerances are rounding counts: an output rounded to a type t is off by at
most half a step, H[t] = finfo(t).eps / 2 of its magnitude (bf16 2^-8, fp16
2^-11, float32 2^-24, e4m3 2^-4, e5m2 2^-3); a float32 sum of n terms by at
most n U of the sum of magnitudes, U = 2^-24.  The matrix units' inner sums of
128 products count 2 U a term (they may cut instead of rounding)."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

U = 2.0 ** -24
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
NAMES = {"e4m3": E4, "e5m2": E5}
TOP = {"e4m3": 448.0, "e5m2": 57344.0}
SMALL8 = {"e4m3": 2.0 ** -10, "e5m2": 2.0 ** -17}  # half the smallest step
H = {t: torch.finfo(t).eps / 2 for t in (BF, HF, F32, E4, E5)}
TINY = {BF: 2.0 ** -134, HF: 2.0 ** -25, F32: 2.0 ** -126}  # half a step among the smallest values


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


def gen(dev, seed):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return g


def randn(dev, seed, *shape):
    return torch.randn(*shape, generator=gen(dev, seed), device=dev)


def strided(x, ld, fill=float("nan")):
    """x in rows `ld` elements apart, the gaps filled with NaN."""
    big = torch.full((x.shape[0], ld), fill, dtype=torch.float32, device=x.device).to(x.dtype)
    big[:, : x.shape[1]] = x
    return big[:, : x.shape[1]]


def shifted(x):
    """x at one element past a 16-byte boundary, rows packed."""
    flat = torch.zeros(x.numel() + 1, dtype=x.dtype, device=x.device)
    flat[1:] = x.reshape(-1)
    return flat[1:].view(x.shape)


def within(got, want, tol, what=""):
    d = (got.double() - want).abs()
    bad = ~(d <= tol)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((d / tol).nan_to_num(1e9).max()):.3g} x tolerance"


def spread(s, rows, cols, square):
    s = s.double().repeat_interleave(128, 1)[:, :cols]
    return s.repeat_interleave(128, 0)[:rows] if square else s


def check_eight(q, s, y, eight, square, y_tol):
    """q, s against the values y (known to y_tol, absolute): the scale is the block's largest magnitude over the
    type's largest value, every value within half a step of y."""
    m, n = y.shape
    tall = 128 if square else 1
    pad = torch.zeros((m + tall - 1) // tall * tall, (n + 127) // 128 * 128, dtype=torch.float64, device=y.device)
    pad[:m, :n] = y.abs()
    slack = torch.zeros_like(pad)
    slack[:m, :n] = y_tol
    shape = (pad.shape[0] // tall, tall, pad.shape[1] // 128, 128)
    want = pad.view(shape).amax((1, 3)).clamp_min(2.0 ** -100) / TOP[eight]
    assert s.shape == want.shape
    within(s, want, want * 2 * U + slack.view(shape).amax((1, 3)) / TOP[eight], "scale")
    sc = spread(s, m, n, square)
    back = q.double() * sc
    # half a step of y, half the smallest step, and y's own error; 4 U for the float32 quotient
    within(back, y, y.abs() * (H[NAMES[eight]] + 4 * U) + sc * SMALL8[eight] + 2 * y_tol, "8-bit values")


# ------------------------------------------------------------------- norm
NORM_SHAPES = [(1, 1), (1, 8), (1, 1024), (3, 127), (5, 128), (7, 129), (2, 504), (33, 520), (65, 1000), (9, 1337),
               (4, 2048), (6, 2056), (3, 4096), (2, 4097), (3, 8192), (2, 9000), (2, 16384), (1, 16383), (300, 640),
               (2500, 136)]


def norm_reference(h, w, eps):
    h = h.double()
    rstd = (h.square().mean(1) + eps) ** -0.5
    return rstd, h * rstd[:, None] * w.double()


# a row's mean of squares: at most 64 additions in a lane, 6 across a wave and 16 across waves, the division and eps;
# half of that after the root, and the root, the reciprocal and the two products
def rstd_tol():
    return (64 + 6 + 16 + 4) / 2 * U + 4 * U


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("rows, width", NORM_SHAPES)
def test_norm_forward(dev, rows, width, t):
    x = randn(dev, 1, rows, width).mul_(3).to(t)
    r = randn(dev, 2, rows, width).to(t)
    w = 1 + 0.2 * randn(dev, 3, width)
    for eight, res, w_ in (("e4m3", r, w), ("e5m2", None, w.to(t)), (None, r, w.to(t))):
        out = mr.rms_norm_forward(x, w_, 1e-5, residual=res, eight=eight)
        if res is None:
            assert out.h is x
        else:
            want = x.double() + r.double()
            within(out.h, want, want.abs() * (H[t] + U) + TINY[t], "h")
        rstd, y = norm_reference(out.h, w_, 1e-5)
        within(out.rstd, rstd, rstd * rstd_tol(), "rstd")
        f32_tol = y.abs() * (rstd_tol() + 2 * U)
        within(out.y, y, y.abs() * H[t] * 1.01 + f32_tol + TINY[t], "y")
        if eight:
            check_eight(out.q, out.scales, y, eight, False, f32_tol)
        else:
            assert out.q is None and out.scales is None


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows, width", [(5, 1024), (3, 333), (4, 4096)])
def test_norm_strides_and_alignment(dev, rows, width, t):
    x, r = randn(dev, 4, rows, width).to(t), randn(dev, 5, rows, width).to(t)
    w = 1 + 0.2 * randn(dev, 6, width)
    want = mr.rms_norm_forward(x, w, 1e-6, residual=r, eight="e4m3")
    for lay in (lambda v: strided(v, width + 24), lambda v: strided(v, width + 3), shifted):
        got = mr.rms_norm_forward(lay(x), w, 1e-6, residual=lay(r), eight="e4m3")
        assert torch.equal(got.h, want.h)
        rstd, y = norm_reference(want.h, w, 1e-6)
        within(got.y, y, y.abs() * (H[t] * 1.01 + rstd_tol() + 2 * U) + TINY[t])
        check_eight(got.q, got.scales, y, "e4m3", False, y.abs() * (rstd_tol() + 2 * U))
        dy = randn(dev, 7, rows, width).to(t)
        a, da = mr.rms_norm_backward(dy, want.h, want.rstd, w, dresidual=r)
        b, db = mr.rms_norm_backward(lay(dy), lay(want.h), want.rstd, w, dresidual=lay(r))
        tol = a.double().abs().max() * (2 * H[t] + 200 * U) + 1e-30
        within(b, a.double(), tol)
        within(db, da.double(), da.double().abs().max() * 100 * U + 1e-6)


def test_norm_rows_keep_to_themselves(dev):
    """A NaN row, an infinite row, a zero row: the others are as without them."""
    x = randn(dev, 8, 6, 256).to(BF)
    w = torch.ones(256, device=dev)
    want = mr.rms_norm_forward(x, w, 1e-6, eight="e4m3")
    y = x.clone()
    y[1, 7] = float("nan")
    y[3, 9] = float("inf")
    y[4] = 0
    got = mr.rms_norm_forward(y, w, 1e-6, eight="e4m3")
    keep = [0, 2, 5]
    assert torch.equal(got.y[keep], want.y[keep]) and torch.equal(got.scales[keep], want.scales[keep])
    assert bool(got.y[1].isnan().all()) and bool(got.rstd[1].isnan()) and bool(got.scales[1].isnan().all())
    assert got.rstd[3] == 0 and bool(got.y[3, 9].isnan()) and bool((got.y[3, :9] == 0).all())
    assert bool((got.y[4] == 0).all()) and bool((got.q[4].float() == 0).all()) and bool((got.scales[4] > 0).all())
    assert float(got.rstd[4]) == pytest.approx(1e3, rel=1e-6)


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("rows, width", [s for s in NORM_SHAPES if s[1] > 1])
def test_norm_backward(dev, rows, width, t):
    h = randn(dev, 11, rows, width).mul_(2).to(t)
    dy = randn(dev, 12, rows, width).to(t)
    res = randn(dev, 13, rows, width).to(t)
    w = 1 + 0.2 * randn(dev, 14, width)
    rstd = norm_reference(h, w, 1e-6)[0].float()
    for dres, w_ in ((res, w), (None, w.to(t))):
        dx, dw = mr.rms_norm_backward(dy, h, rstd, w_, dresidual=dres)
        xh = h.double() * rstd.double()[:, None]
        g = dy.double() * w_.double()
        c = (g * xh).mean(1, keepdim=True)
        core = rstd.double()[:, None] * (g - xh * c)
        want = core + (dres.double() if dres is not None else 0)
        # c: a lane's at most 64 additions and 22 across lanes, 3 roundings of a term; then 4 roundings of each part
        c_tol = 90 * U * (g * xh).abs().mean(1, keepdim=True)
        part = rstd.double()[:, None] * (xh.abs() * (c_tol + 4 * U * c.abs()) + 4 * U * g.abs())
        within(dx, want, want.abs() * (H[t] * 1.01 + U) + part + TINY[t], "dx")
        terms = (dy.double() * xh)
        # a lane adds its rows one by one, then at most 4 waves and 512 workgroups are joined
        n = min(rows, max(rows // 512 + 2, 2)) + 4 + 512 // 4 + 8
        within(dw, terms.sum(0), n * U * terms.abs().sum(0) + 1e-30, "dweight")
    assert mr.rms_norm_backward(dy, h, rstd, w, weight_grad=False)[1] is None


def test_norm_gradient_is_the_slope(dev):
    """Against differences of the 64-bit forward formula: f = sum(y c)."""
    rows, width, eps = 3, 200, 1e-4
    h = randn(dev, 15, rows, width)
    c = randn(dev, 16, rows, width)
    w = 1 + 0.2 * randn(dev, 17, width)
    rstd = norm_reference(h, w, eps)[0].float()
    dx, dw = mr.rms_norm_backward(c, h, rstd, w)
    e = 1e-5
    for k in range(6):
        v = randn(dev, 20 + k, rows, width).double()
        u = randn(dev, 30 + k, width).double()

        def f(s):
            return float((norm_reference(h.double() + s * v, w.double() + s * u, eps)[1] * c.double()).sum())

        slope = (f(e) - f(-e)) / (2 * e)
        got = float((dx.double() * v).sum() + (dw.double() * u).sum())
        # e^2 of the third derivative, 2^-53 / e of the values, float32 gradients
        scale = float((dx.double() * v).abs().sum() + (dw.double() * u).abs().sum())
        assert abs(got - slope) <= scale * 1e-5, (got, slope)


def test_norm_without_rows(dev):
    x = torch.zeros(0, 64, dtype=BF, device=dev)
    w = torch.ones(64, device=dev)
    out = mr.rms_norm_forward(x, w, 1e-6, residual=x, eight="e4m3")
    assert out.y.shape == (0, 64) and out.scales.shape == (0, 1)
    dx, dw = mr.rms_norm_backward(x, x, out.rstd, w)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


# --------------------------------------------------------------- quantise
@pytest.mark.parametrize("eight", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", ["vector", "square"])
@pytest.mark.parametrize("m, n, t", [(1, 1, F32), (1, 1000, BF), (127, 129, BF), (128, 128, F32), (130, 257, HF),
                                     (300, 64, BF), (257, 8, F32), (1000, 392, BF), (64, 2049, HF)])
def test_quantize(dev, m, n, t, block, eight):
    x = (randn(dev, 41, m, n) * torch.exp(2 * randn(dev, 42, m, 1))).to(t)
    x[:, n // 2] *= 0
    both = mr.quantize_blocks(x, eight, block=block, order="both")
    square = block == "square"
    zero = torch.zeros((), dtype=torch.float64, device=dev)
    check_eight(both.q, both.scales, x.double(), eight, square, zero)
    check_eight(both.qt, both.scales_t, x.double().t(), eight, square, zero)
    if square:
        assert torch.equal(both.scales_t, both.scales.t())
        assert torch.equal(both.qt.float(), both.q.float().t())
    rows, cols = mr.quantize_blocks(x, eight, block=block), mr.quantize_blocks(x, eight, block=block, order="columns")
    assert rows.qt is None and cols.q is None
    assert torch.equal(rows.q.float(), both.q.float()) and torch.equal(rows.scales, both.scales)
    assert torch.equal(cols.qt.float(), both.qt.float()) and torch.equal(cols.scales_t, both.scales_t)
    for lay in (lambda v: strided(v, n + 5), lambda v: strided(v, (n + 31) // 16 * 16), shifted):
        other = mr.quantize_blocks(lay(x), eight, block=block, order="both")
        assert torch.equal(other.q.float(), both.q.float()) and torch.equal(other.qt.float(), both.qt.float())
        assert torch.equal(other.scales, both.scales) and torch.equal(other.scales_t, both.scales_t)


def test_quantize_special_values(dev):
    x = randn(dev, 43, 256, 384)
    x[3, 130] = float("nan")
    x[200, 5] = float("-inf")
    x[130, 256:] = 0
    x[131, 256:] = 1e-42  # below every normal float32
    q = mr.quantize_blocks(x, "e4m3", order="both")
    back = q.q.float() * q.scales.repeat_interleave(128, 1)
    hit = torch.zeros(256, 384, dtype=torch.bool, device=dev)
    hit[3, 128:256] = hit[200, :128] = True
    assert torch.equal(back.isnan(), hit)
    assert bool((back[130:132, 256:] == 0).all())
    back_t = q.qt.float() * q.scales_t.repeat_interleave(128, 1)
    hit_t = torch.zeros(384, 256, dtype=torch.bool, device=dev)
    hit_t[130, :128] = hit_t[5, 128:] = True
    assert torch.equal(back_t.isnan(), hit_t)


# ---------------------------------------------------------------- product
def operand(dev, seed, rows, k, eight, square):
    x = randn(dev, seed, rows, k) * torch.exp(randn(dev, seed + 1, rows, 1))
    r = mr.quantize_blocks(x, eight, block="square" if square else "vector")
    return r.q, r.scales


def product_reference(a, sa, b, sb):
    m, k = a.shape
    n = b.shape[0]
    x = a.double() * spread(sa, m, k, sa.shape[0] != m)
    y = b.double() * spread(sb, n, k, sb.shape[0] != n)
    return x @ y.t().contiguous(), x.abs() @ y.abs().t().contiguous()


def product_tol(want, mag, k, out_t, extra=0):
    # 128 products of a block at 2 U, the blocks' scaled sums and the scale's roundings, up to 16 splits joined
    n = 2 * 128 + (k + 127) // 128 + 3 + 16 + extra
    return mag * n * U + want.abs() * H[out_t] * 1.01 + TINY[out_t]


PRODUCTS = [(1, 16, 128), (1, 1, 1), (5, 33, 129), (16, 256, 1024), (17, 100, 300), (33, 64, 2048), (64, 130, 257),
            (65, 129, 255), (128, 128, 128), (100, 1000, 640), (300, 260, 1920), (256, 384, 8192), (129, 4096, 96),
            (4100, 4100, 200)]


@pytest.mark.parametrize("a8", ["e4m3", "e5m2"])
@pytest.mark.parametrize("b_square", [False, True])
@pytest.mark.parametrize("m, n, k", PRODUCTS)
def test_product(dev, m, n, k, b_square, a8):
    a, sa = operand(dev, 51, m, k, a8, False)
    b, sb = operand(dev, 61, n, k, "e4m3", b_square)
    want, mag = product_reference(a, sa, b, sb)
    for t in (BF, HF, F32):
        got = mr.block_scaled_matmul(a, sa, b, sb, out_dtype=t)
        ref = want.clamp(-65504, 65504) if t == HF else want
        within(got.clamp(-65504, 65504) if t == HF else got, ref, product_tol(ref, mag, k, t), f"{t}")
    again = mr.block_scaled_matmul(a, sa, b, sb, out_dtype=F32)
    assert torch.equal(again, got)


def test_product_square_scales_of_both(dev):
    m, n, k = 300, 200, 400
    a, sa = operand(dev, 71, m, k, "e4m3", True)
    b, sb = operand(dev, 72, n, k, "e4m3", True)
    want, mag = product_reference(a, sa, b, sb)
    within(mr.block_scaled_matmul(a, sa, b, sb, out_dtype=F32), want, product_tol(want, mag, k, F32))


@pytest.mark.parametrize("m, n, k", [(8, 100, 300), (200, 150, 300), (300, 200, 4096)])
def test_product_strides_accumulation_and_edges(dev, m, n, k):
    """Operands with NaN between their rows and past their end, odd alignments, results into part of a larger matrix."""
    a, sa = operand(dev, 73, m, k, "e4m3", False)
    b, sb = operand(dev, 74, n, k, "e4m3", False)
    want, mag = product_reference(a, sa, b, sb)
    base = mr.block_scaled_matmul(a, sa, b, sb, out_dtype=F32)
    for lay in (lambda v: strided(v, k + 7), lambda v: strided(v, (k + 47) // 16 * 16), shifted):
        got = mr.block_scaled_matmul(lay(a), strided(sa, sa.shape[1] + 2), lay(b), strided(sb, sb.shape[1] + 1), out_dtype=F32)
        assert torch.equal(got, base)
    c = randn(dev, 75, m, n + 9)
    keep = c.clone()
    mr.block_scaled_matmul(a, sa, b, sb, out=c[:, 3:3 + n], accumulate=True)
    assert torch.equal(c[:, :3], keep[:, :3]) and torch.equal(c[:, 3 + n:], keep[:, 3 + n:])
    total = want + keep[:, 3:3 + n].double()
    within(c[:, 3:3 + n], total, product_tol(total, mag, k, F32, 2) + U * keep[:, 3:3 + n].double().abs())
    mr.block_scaled_matmul(a, sa, b, sb, out=c[:, 3:3 + n])
    assert torch.equal(c[:, 3:3 + n], base)


def test_product_nan_reaches_its_row_and_column_only(dev):
    m, n, k = 200, 150, 300
    a, sa = operand(dev, 76, m, k, "e4m3", False)
    b, sb = operand(dev, 77, n, k, "e4m3", False)
    base = mr.block_scaled_matmul(a, sa, b, sb, out_dtype=F32)
    sa, sb = sa.clone(), sb.clone()
    sa[17, 1] = float("nan")
    sb[3, 2] = float("inf")
    got = mr.block_scaled_matmul(a, sa, b, sb, out_dtype=F32)
    hit = torch.zeros(m, n, dtype=torch.bool, device=dev)
    hit[17] = True
    assert bool(got[17].isnan().all())
    fine = torch.ones(m, n, dtype=torch.bool, device=dev)
    fine[17] = False
    fine[:, 3] = False
    assert torch.equal(got[fine], base[fine]) and not bool(got[:, 3].isfinite().any())


def test_layer_products_through_the_quantiser(dev):
    """Y = X W^T, dX = dY W, dW = dY^T X on one quantisation of each operand, against the products of the values it kept."""
    T, N, K = 333, 260, 384
    x, w, dy = randn(dev, 78, T, K).to(BF), randn(dev, 79, N, K), randn(dev, 80, T, N).to(BF)
    qx, qw, qd = (mr.quantize_blocks(v, "e4m3", block=b, order="both") for v, b in ((x, "vector"), (w, "square"), (dy, "vector")))
    for a, sa, b, sb, k in ((qx.q, qx.scales, qw.q, qw.scales, K), (qd.q, qd.scales, qw.qt, qw.scales_t, N),
                            (qd.qt, qd.scales_t, qx.qt, qx.scales_t, T)):
        want, mag = product_reference(a, sa, b, sb)
        within(mr.block_scaled_matmul(a, sa, b, sb, out_dtype=F32), want, product_tol(want, mag, k, F32))
    full = dy.double().t().contiguous() @ x.double()
    got = mr.block_scaled_matmul(qd.qt, qd.scales_t, qx.qt, qx.scales_t, out_dtype=F32).double()
    # both operands are off by at most 2^-4 of each value
    bound = 2.2 * 2.0 ** -4 * (dy.double().abs().t().contiguous() @ x.double().abs())
    within(got, full, bound + 1.0)


def test_product_without_rows(dev):
    b, sb = operand(dev, 81, 64, 128, "e4m3", True)
    a = torch.zeros(0, 128, device=dev).to(E4)
    assert mr.block_scaled_matmul(a, torch.zeros(0, 1, device=dev), b, sb).shape == (0, 64)


# ---------------------------------------------------------------- grouped
def grouped_reference(x, w, off, transpose):
    y = torch.zeros(x.shape[0], w.shape[2 if transpose else 1], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    for e in range(w.shape[0]):
        s = slice(off[e], off[e + 1])
        we = w[e].double() if transpose else w[e].double().t().contiguous()
        y[s] = x[s].double() @ we
        mag[s] = x[s].double().abs() @ we.abs()
    return y, mag


def grouped_weight_reference(dy, x, off):
    E = len(off) - 1
    d = torch.zeros(E, dy.shape[1], x.shape[1], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(d)
    for e in range(E):
        s = slice(off[e], off[e + 1])
        d[e] = dy[s].double().t().contiguous() @ x[s].double()
        mag[e] = dy[s].double().abs().t().contiguous() @ x[s].double().abs()
    return d, mag


GROUPS = [
    ([0, 1], 8, 8), ([0, 3], 5, 7), ([0, 0, 0, 16], 128, 128), ([0, 5, 5, 130, 131], 96, 160),
    ([2, 2, 9, 300], 130, 72), ([0, 256, 512, 513], 264, 320), ([1, 200, 200, 200, 391], 100, 1001),
    ([0] * 40 + [70] * 30 + [129], 72, 136), ([7, 500], 257, 129), ([0, 127, 255, 384, 1000], 384, 64),
]


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("case", range(len(GROUPS)))
def test_grouped(dev, case, t):
    off, n, k = GROUPS[case]
    rows = off[-1] + case % 3 * 5  # some rows past the last expert
    E = len(off) - 1
    x, w, dy = randn(dev, 91, rows, k).to(t), randn(dev, 92, E, n, k).to(t), randn(dev, 93, rows, n).to(t)
    for o in (torch.tensor(off, dtype=torch.int32, device=dev), torch.tensor(off, dtype=torch.int64, device=dev)):
        for src, tr, steps in ((x, False, k), (dy, True, n)):
            want, mag = grouped_reference(src, w, off, tr)
            for out in (t, F32):
                got = mr.grouped_matmul(src, w, o, transpose=tr, out_dtype=out)
                ref = want.clamp(-65504, 65504) if out == HF else want
                within(got.clamp(-65504, 65504) if out == HF else got, ref,
                       mag * 2 * (steps + 1) * U + ref.abs() * H[out] * 1.01 + TINY[out], f"transpose {tr} {out}")
                outside = torch.ones(rows, dtype=torch.bool, device=dev)
                outside[off[0]:off[-1]] = False
                assert bool((got[outside] == 0).all())
        want, mag = grouped_weight_reference(dy, x, off)
        most = max(off[e + 1] - off[e] for e in range(E))
        got = mr.grouped_weight_grad(dy, x, o)
        within(got, want, mag * 2 * (most + 1) * U + want.abs() * U, "weights")
        again = mr.grouped_weight_grad(dy, x, o)
        assert torch.equal(got, again)
        half = mr.grouped_weight_grad(dy, x, o, out_dtype=t)
        ref = want.clamp(-65504, 65504)
        within(half.clamp(-65504, 65504), ref, mag * 2 * (most + 1) * U + ref.abs() * H[t] * 1.01 + TINY[t])
        for e in range(E):
            if off[e] == off[e + 1]:
                assert bool((got[e] == 0).all())


@pytest.mark.parametrize("n, k", [(96, 160), (100, 77)])
def test_grouped_strides_and_neighbours(dev, n, k):
    """Strided and unaligned operands; NaN in the gaps, in rows of no expert and in other experts' rows stays there."""
    off = [3, 40, 40, 177, 200]
    rows, E = 210, 4
    o = torch.tensor(off, dtype=torch.int32, device=dev)
    x, w, dy = randn(dev, 94, rows, k).to(BF), randn(dev, 95, E, n, k).to(BF), randn(dev, 96, rows, n).to(BF)
    y, dx, dw = mr.grouped_matmul(x, w, o), mr.grouped_matmul(dy, w, o, transpose=True), mr.grouped_weight_grad(dy, x, o)
    for v in (x, dy):
        v[:3] = float("nan")
        v[200:] = float("inf")
    for lay in (lambda v: strided(v, v.shape[1] + 11), lambda v: strided(v, (v.shape[1] + 23) // 8 * 8), shifted):
        big = torch.full((E + 1, n + 2, k + 8 - k % 8), float("nan"), device=dev).to(BF)
        ws = big[:E, :n, :k]
        ws.copy_(w)
        assert torch.equal(mr.grouped_matmul(lay(x), ws, o), y)
        assert torch.equal(mr.grouped_matmul(lay(dy), ws, o, transpose=True), dx)
        assert torch.equal(mr.grouped_weight_grad(lay(dy), lay(x), o), dw)
    bank = torch.zeros(E, n + 3, k + 5, device=dev)
    mr.grouped_weight_grad(dy, x, o, out=bank[:, 1:1 + n, 2:2 + k])
    assert torch.equal(bank[:, 1:1 + n, 2:2 + k], dw)
    mr.grouped_weight_grad(dy, x, o, out=bank[:, 1:1 + n, 2:2 + k], accumulate=True)
    assert torch.equal(bank[:, 1:1 + n, 2:2 + k], dw + dw)
    bank[:, 1:1 + n, 2:2 + k] = 0
    assert bool((bank == 0).all())
    x[50, :] = float("nan")  # expert 2
    got = mr.grouped_matmul(x, w, o)
    assert bool(got[50].isnan().all()) and torch.equal(got[51:200], y[51:200]) and torch.equal(got[3:50], y[3:50])
    got = mr.grouped_weight_grad(dy, x, o)
    assert bool(got[2].isnan().all()) and torch.equal(got[[0, 1, 3]], dw[[0, 1, 3]])


def test_grouped_without_rows(dev):
    o = torch.zeros(4, dtype=torch.int32, device=dev)
    x, w = torch.zeros(0, 16, dtype=BF, device=dev), randn(dev, 97, 3, 24, 16).to(BF)
    assert mr.grouped_matmul(x, w, o).shape == (0, 24)
    d = mr.grouped_weight_grad(torch.zeros(0, 24, dtype=BF, device=dev), x, o)
    assert d.shape == (3, 24, 16) and bool((d == 0).all())
    y = mr.grouped_matmul(randn(dev, 98, 50, 16).to(BF), w, o)
    assert bool((y == 0).all())


def test_grouped_offsets_out_of_range_are_clamped(dev):
    """Offsets past the rows count as the last row: nothing out of range is read or written."""
    x, w = randn(dev, 99, 40, 64).to(BF), randn(dev, 100, 2, 48, 64).to(BF)
    o = torch.tensor([-5, 10, 1000], dtype=torch.int32, device=dev)
    good = torch.tensor([0, 10, 40], dtype=torch.int32, device=dev)
    dy = randn(dev, 101, 40, 48).to(BF)
    assert torch.equal(mr.grouped_matmul(x, w, o), mr.grouped_matmul(x, w, good))
    assert torch.equal(mr.grouped_weight_grad(dy, x, o), mr.grouped_weight_grad(dy, x, good))


# -------------------------------------------------- far rows, streams, graphs
def test_rows_past_32_bits(dev):
    """Rows whose element offsets pass 2^31 (and byte offsets 2^32)."""
    rows, width = 270001, 8192
    x = torch.zeros(rows, width, dtype=BF, device=dev)
    tail = randn(dev, 111, 200, width).to(BF)
    x[-200:] = tail
    w = torch.ones(width, device=dev)
    got, want = mr.rms_norm_forward(x, w, 1e-6, eight="e4m3"), mr.rms_norm_forward(tail, w, 1e-6, eight="e4m3")
    assert torch.equal(got.y[-200:], want.y) and torch.equal(got.q[-200:].float(), want.q.float())
    dx, dw = mr.rms_norm_backward(x, x, got.rstd, w)
    d2, _ = mr.rms_norm_backward(tail, tail, want.rstd, w)
    assert torch.equal(dx[-200:], d2)
    del dx
    wts = randn(dev, 112, 1, 64, width).to(BF)
    o = torch.tensor([rows - 200, rows], dtype=torch.int64, device=dev)
    o2 = torch.tensor([0, 200], dtype=torch.int64, device=dev)
    y = mr.grouped_matmul(x, wts, o)
    assert torch.equal(y[-200:], mr.grouped_matmul(tail, wts, o2)) and bool((y[:-200] == 0).all())
    q = mr.quantize_blocks(x)
    q2 = mr.quantize_blocks(tail)
    assert torch.equal(q.q[-200:].float(), q2.q.float())
    b, sb = operand(dev, 113, 64, width, "e4m3", True)
    c = mr.block_scaled_matmul(q.q, q.scales, b, sb, out_dtype=F32)
    c2 = mr.block_scaled_matmul(q2.q, q2.scales, b, sb, out_dtype=F32)
    # two tile shapes may add in another order
    ref, mag = product_reference(q2.q, q2.scales, b, sb)
    within(c[-200:], ref, product_tol(ref, mag, width, F32))
    within(c2, ref, product_tol(ref, mag, width, F32))


def step(x, res, w, W8, off, bank):
    """One pass through the operators as a layer uses them."""
    n = mr.rms_norm_forward(x, w, 1e-6, residual=res, eight="e4m3")
    y = mr.block_scaled_matmul(n.q, n.scales, W8.q, W8.scales)
    z = mr.grouped_matmul(y, bank, off)
    dy = mr.grouped_matmul(z, bank, off, transpose=True)
    dbank = mr.grouped_weight_grad(z, y, off)
    q = mr.quantize_blocks(dy, "e5m2", order="both")
    dn = mr.block_scaled_matmul(q.q, q.scales, W8.qt, W8.scales_t)
    xt = mr.quantize_blocks(n.y, order="columns")
    dW = mr.block_scaled_matmul(q.qt, q.scales_t, xt.qt, xt.scales_t, out_dtype=F32)
    dx, dw = mr.rms_norm_backward(dn, n.h, n.rstd, w, dresidual=x)
    return [n.h, n.y, y, z, dbank, dW, dx, dw]


def step_inputs(dev, seed):
    T, D, N, E = 600, 512, 384, 5
    sizes = torch.tensor([0, 100, 0, 331, 150], device=dev)
    off = torch.cat([torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(sizes, 0)])
    x, res = randn(dev, seed, T, D).to(BF), randn(dev, seed + 1, T, D).to(BF)
    W8 = mr.quantize_blocks(randn(dev, seed + 2, N, D) / 20, "e4m3", block="square", order="both")
    return x, res, 1 + 0.1 * randn(dev, seed + 3, D), W8, off, (randn(dev, seed + 4, E, 256, N) / 20).to(BF)


def test_other_streams(dev):
    args = step_inputs(dev, 120)
    want = step(*args)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = step(*args)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    n = mr.rms_norm_forward(args[0], args[2], 1e-6, residual=args[1], eight="e4m3", stream=s)
    s.synchronize()
    assert torch.equal(n.h, want[0]) and torch.equal(n.y, want[1])


def test_graph_replays(dev):
    """A captured pass gives the eager results under new inputs and new group sizes, replay after replay."""
    x, res, w, W8, off, bank = step_inputs(dev, 130)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(x, res, w, W8, off, bank)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(x, res, w, W8, off, bank)
    for k in range(4):
        x.copy_(randn(dev, 140 + k, *x.shape).to(BF))
        sizes = [[0, 100, 0, 331, 150], [600, 0, 0, 0, 0], [1, 2, 3, 4, 5], [120, 120, 120, 120, 120]][k]
        off[1:] = torch.cumsum(torch.tensor(sizes, device=dev), 0)
        g.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in out]
        for a, b in zip(got, step(x, res, w, W8, off, bank)):
            assert torch.equal(a, b)
        torch.cuda.synchronize()
