"""The operators around a bank of experts on the GPU against plain 64-bit formulas.

Tolerances count roundings: U = 2^-24 for a float32 operation, H[t] =
finfo(t).eps / 2 for an output rounded to t, exp and log 2 U of themselves, a
float32 sum of n terms n U of the sum of magnitudes.  Whole numbers and copies
have to be equal."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

from test_gpu_linear import BF, F32, H, HF, TINY, U, gen, randn, shifted, strided, within  # noqa: E402

INF = math.inf


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


# ---------------------------------------------------------------- routing
def chosen_of(l, k):
    """The k largest of each row, first of equals first, -1 where only -inf is left."""
    left = l.double().clone()
    number = torch.arange(l.shape[1], device=l.device)
    out = []
    for _ in range(k):
        peak = left.max(1, keepdim=True).values
        first = torch.where(left == peak, number, l.shape[1]).min(1).values
        out.append(torch.where(peak[:, 0] == -INF, -1, first))
        left[torch.arange(l.shape[0], device=l.device), first] = -INF
    return torch.stack(out, 1)


def check_route(logits, k, normalize):
    r = mr.route_tokens(logits, k, normalize=normalize)
    tokens, experts = logits.shape
    assert r.experts.shape == (tokens, k) and r.experts.dtype == torch.int32
    want = chosen_of(logits, k)
    assert torch.equal(r.experts.long(), want)
    l = logits.double()
    v = torch.where(want >= 0, l.gather(1, want.clamp_min(0)), -INF)
    s = v if normalize else l
    top = v[:, :1]
    empty = top[:, 0] == -INF
    safe = torch.where(empty[:, None], 0.0, top)
    total = torch.exp(s - safe).sum(1)
    log_sum = safe[:, 0] + torch.log(total)
    # exp of a rounded difference, the sum's additions, the quotient
    n = 4 * math.ceil(experts / 64) + 10
    w = torch.where(empty[:, None], 0.0, torch.exp(v - safe) / total[:, None])
    spread = torch.where(v == -INF, 0.0, safe - v)
    rest = torch.where(s == -INF, 0.0, (safe - s) * torch.exp(s - safe)).sum(1, keepdim=True) / total.clamp_min(1e-300)[:, None]
    tol = w * (spread + rest + n + 8) * 2 * U + 2.0 ** -126
    within(r.weights, w, tol, "weights")
    assert torch.equal(r.log_sum[empty], torch.full_like(r.log_sum[empty], -INF))
    l_tol = (safe.abs()[:, 0] + torch.log(total).abs() + 1) * 4 * U + (rest[:, 0] + n) * 2 * U
    within(r.log_sum[~empty], log_sum[~empty], l_tol[~empty], "log_sum")
    return r


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("tokens, experts, k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (17, 16, 16), (8, 64, 8), (33, 65, 6),
                                                (100, 128, 1), (15, 130, 7), (64, 256, 8), (16, 257, 4), (7, 384, 8),
                                                (5, 385, 3), (9, 512, 16), (6, 513, 8), (3, 1000, 9), (2, 1025, 2),
                                                (4, 2048, 16), (5, 2051, 8), (2, 4096, 16), (3000, 12, 2)])
def test_route(dev, tokens, experts, k, t):
    logits = randn(dev, experts, tokens, experts).mul_(2).to(t)
    for normalize in (True, False):
        check_route(logits, k, normalize)


@pytest.mark.parametrize("experts, k", [(8, 3), (64, 8), (300, 16), (700, 5)])
def test_route_ties_go_to_the_lowest(dev, experts, k):
    g = gen(dev, 1)
    logits = torch.randint(-2, 3, (50, experts), generator=g, device=dev).float()
    logits[0], logits[1, ::2], logits[2] = 0.0, -0.0, -1e30
    logits[1, 1::2] = 0.0  # the zeros are one value
    for t in (F32, BF):
        check_route(logits.to(t), k, True)
        check_route(logits.to(t), k, False)


@pytest.mark.parametrize("experts", [64, 128, 250, 256, 384, 512])
@pytest.mark.parametrize("k", [3, 8])
def test_route_many_that_reach(dev, experts, k):
    """Each count of logits that reach the k-th of the lanes' largest, from k to 60:
    they stand in the columns of k lanes of 16, one of which holds the lowest alone."""
    g = torch.Generator().manual_seed(experts + k)
    rows = []
    for count in range(k, 61):
        lanes = torch.randperm(16, generator=g)[:k].tolist()
        of = [[c for c in range(experts) if c // 4 % 16 == lane] for lane in lanes]
        row = torch.rand(experts, generator=g) - 5.0
        row[of[0][0]] = 4.0
        rest = [c for one in of[1:] for c in one[1:]]
        more = [one[0] for one in of[1:]] + [rest[i] for i in torch.randperm(len(rest), generator=g).tolist()]
        at = more[: count - 1]
        row[at] = 4.0 + torch.rand(len(at), generator=g)
        rows.append(row)
    logits = torch.stack(rows).to(dev)
    for t in (F32, HF, BF):
        for normalize in (True, False):
            check_route(logits.to(t), k, normalize)


@pytest.mark.parametrize("experts, k", [(8, 3), (64, 8), (300, 16), (700, 5)])
def test_route_masked(dev, experts, k):
    """Experts at -inf and at the type's lowest value; tokens with fewer than k experts, with one, with none."""
    for t in (F32, BF, HF):
        logits = randn(dev, 3, 40, experts).to(t)
        logits[0] = -INF
        logits[1] = -INF
        logits[1, experts // 2] = 3.0
        logits[2, : experts - 2] = -INF
        logits[3] = torch.finfo(t).min
        logits[4, 1:] = torch.finfo(t).min
        logits[5:20][torch.rand(15, experts, generator=gen(dev, 4), device=dev) < 0.7] = -INF
        for normalize in (True, False):
            r = check_route(logits, k, normalize)
            assert bool((r.experts[0] == -1).all()) and bool((r.weights[0] == 0).all())
            assert r.experts[1].tolist() == [experts // 2] + [-1] * (k - 1) and r.weights[1].tolist() == [1.0] + [0.0] * (k - 1)
            d = mr.route_tokens_backward(randn(dev, 5, 40, k), logits, r, normalize=normalize)
            assert bool(torch.isfinite(d).all())
            assert bool((d[logits == -INF] == 0).all())


def test_route_values_that_are_no_numbers(dev):
    logits = randn(dev, 3, 6, 20)
    logits[1, 7], logits[2, 9], logits[3, 0], logits[3, 5] = math.nan, INF, -INF, 1e38
    logits[4, 2], logits[4, 3] = INF, math.nan
    for normalize in (True, False):
        r = mr.route_tokens(logits, 4, normalize=normalize)
        assert int(r.experts[1, 0]) == 7 and int(r.experts[2, 0]) == 9 and r.experts[4, :2].tolist() == [2, 3]
        for row in r.experts.tolist():
            assert len(set(row)) == 4 and all(0 <= e < 20 for e in row)
        assert bool(r.weights[[1, 2, 4]].isnan().all()) and bool(torch.isfinite(r.weights[[0, 3, 5]]).all())


def test_route_strides(dev):
    logits = randn(dev, 3, 30, 100)
    want = mr.route_tokens(logits, 5)
    for lay in (lambda v: strided(v, 128), lambda v: strided(v, 101), shifted):
        got = mr.route_tokens(lay(logits), 5)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    none = mr.route_tokens(logits[:0], 5)
    assert none.experts.shape == (0, 5)
    assert mr.route_tokens_backward(none.weights, logits[:0], none).shape == (0, 100)


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("tokens, experts, k", [(1, 1, 1), (3, 5, 5), (8, 64, 8), (33, 65, 6), (16, 257, 4), (7, 384, 8),
                                                (9, 512, 16), (3, 1003, 9), (2, 4096, 16), (3000, 12, 2)])
def test_route_backward(dev, tokens, experts, k, t):
    logits = randn(dev, experts, tokens, experts).to(t)
    dw = randn(dev, 9, tokens, k)
    for normalize in (True, False):
        r = mr.route_tokens(logits, k, normalize=normalize)
        got = mr.route_tokens_backward(dw, logits, r, normalize=normalize)
        assert got.dtype == t
        w, d = r.weights.double(), dw.double()
        c, c_abs = (w * d).sum(1, keepdim=True), (w * d).abs().sum(1, keepdim=True)
        at = r.experts.long()
        if normalize:
            want = torch.zeros(tokens, experts, dtype=torch.float64, device=dev).scatter_add_(1, at, w * (d - c))
            tol = torch.zeros_like(want).scatter_add_(1, at, w * (d.abs() + c_abs) * 8 * U)
        else:
            p = torch.softmax(logits.double(), 1)
            gap = logits.double().max(1, keepdim=True).values - logits.double()
            n = 4 * math.ceil(experts / 256) + 6 + 8  # the sum's additions, exp, the quotients
            want = (-p * c).scatter_add_(1, at, w * d)
            tol = (p * (c_abs * 8 + c.abs() * (gap + (p * gap).sum(1, keepdim=True) + n))).scatter_add_(1, at, (w * d).abs() * 4) * U
        within(got, want, want.abs() * H[t] * 1.01 + tol + TINY[t], f"dlogits {normalize}")


def test_route_backward_against_differences(dev):
    tokens, experts, k = 5, 24, 4
    logits, c = randn(dev, 1, tokens, experts), randn(dev, 2, tokens, k)
    for normalize in (True, False):
        r = mr.route_tokens(logits, k, normalize=normalize)
        got = mr.route_tokens_backward(c, logits, r, normalize=normalize)

        def loss(l):
            v = l.gather(1, r.experts.long())
            return (c.double() * torch.exp(v - torch.logsumexp(v if normalize else l, 1, keepdim=True))).sum()

        for i in range(0, tokens * experts, 3):
            step = torch.zeros(tokens, experts, dtype=torch.float64, device=dev)
            step.view(-1)[i] = 1e-5
            want = float(loss(logits.double() + step) - loss(logits.double() - step)) / 2e-5
            # 64-bit rounding over the step 1e-10, curvature 1e-10, the kernel's 50 U
            assert abs(float(got.view(-1)[i]) - want) < 1e-8 + 50 * U


def test_route_backward_of_choices_that_are_no_experts(dev):
    """Choices of -1 and beyond have no part, whatever their weights and gradients hold; the same expert twice adds up."""
    logits = randn(dev, 1, 3, 10)
    chosen = torch.tensor([[2, -1, 5], [11, 1 << 30, -7], [4, 4, 9]], dtype=torch.int32, device=dev)
    w, d = torch.rand(3, 3, device=dev), randn(dev, 2, 3, 3)
    w[0, 1], d[1, 0] = math.nan, INF
    for normalize in (True, False):
        r = mr.Routed(chosen, w, None)
        got = mr.route_tokens_backward(d, logits, r, normalize=normalize)
        ok = (chosen >= 0) & (chosen < 10)
        wd = torch.where(ok, w * d, 0.0).double()
        c = wd.sum(1, keepdim=True)
        part = torch.where(ok, w.double() * (d.double() - c) if normalize else wd, 0.0)
        want = torch.zeros(3, 10, dtype=torch.float64, device=dev).scatter_add_(1, torch.where(ok, chosen, 0).long(), part)
        if not normalize:
            want -= torch.softmax(logits.double(), 1) * c
        within(got, want, 40 * U * (1 + want.abs()))


@pytest.mark.parametrize("experts", [6, 300])
def test_route_far_from_zero(dev, experts):
    """Equal logits at any level share alike, those at the type's lowest value among them, forward and backward."""
    k = 3
    levels = torch.tensor([0.0, 1e4, -1e30, 1e38, torch.finfo(F32).min], device=dev)
    logits = levels[:, None].expand(-1, experts).contiguous()
    d = randn(dev, 1, 5, k)
    for normalize, n in ((True, k), (False, experts)):
        r = mr.route_tokens(logits, k, normalize=normalize)
        within(r.weights, torch.full((5, k), 1 / n, dtype=torch.float64, device=dev), 4 * U / n)
        got = mr.route_tokens_backward(d, logits, r, normalize=normalize)
        c = d.double().sum(1, keepdim=True) / n
        want = torch.zeros(5, experts, dtype=torch.float64, device=dev) if normalize else (-c / n).expand(-1, experts).clone()
        want[:, :k] += (d.double() - c if normalize else d.double()) / n
        within(got, want, 20 * U * d.double().abs().sum(1, keepdim=True) / n)


# ------------------------------------------------------------------ order
def order_of(experts, n):
    e = experts.reshape(-1).long().cpu()
    e = torch.where((e < 0) | (e >= n), n, e)
    by = torch.sort(e, stable=True).indices
    place = torch.empty_like(by)
    place[by] = torch.arange(by.numel())
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), torch.bincount(e, minlength=n + 1)[:n].cumsum(0)])
    return offsets, place.view(experts.shape)


@pytest.mark.parametrize("tokens, k, n", [(0, 2, 5), (1, 1, 1), (1, 8, 64), (7, 3, 2), (16, 8, 64), (65, 1, 3), (129, 4, 16),
                                          (1000, 6, 255), (2048, 8, 1), (2049, 8, 64), (4096, 4, 384), (4097, 4, 900),
                                          (300, 2, 4096), (9000, 3, 2000), (8192, 8, 4096), (16384, 8, 64), (20011, 7, 17),
                                          (100000, 8, 8), (150000, 8, 300), (3, 64, 7), (300000, 4, 40), (90000, 7, 4000)])
def test_order(dev, tokens, k, n):
    g = gen(dev, tokens + n)
    uneven = (torch.rand(tokens, k, generator=g, device=dev) ** 3 * n).int()
    even = torch.randint(0, n, (tokens, k), generator=g, device=dev, dtype=torch.int32)
    away = torch.where(torch.rand(tokens, k, generator=g, device=dev) < 0.3, -1, even)
    for e in (uneven, away.int(), torch.full_like(even, n - 1), torch.full_like(even, n)):
        got = mr.order_by_expert(e, n)
        offsets, place = order_of(e, n)
        assert got.offsets.dtype == got.place.dtype == torch.int32
        assert torch.equal(got.offsets.cpu().long(), offsets)
        assert torch.equal(got.place.cpu().long(), place)


def test_order_types_and_strides(dev):
    e = torch.randint(-2, 12, (3000, 7), generator=gen(dev, 1), device=dev)
    e[5, 2], e[6, 3] = 1 << 40, -(1 << 40)
    offsets, place = order_of(e, 10)
    wide = torch.full((3000, 11), 3, device=dev)
    wide[:, 2:9] = e
    narrow = e.clamp(-3, 1 << 20).int()
    for v in (e, wide[:, 2:9], narrow, torch.cat([narrow] * 2, 1)[:, 7:]):
        got = mr.order_by_expert(v, 10)
        assert torch.equal(got.offsets.cpu().long(), offsets) and torch.equal(got.place.cpu().long(), place)


# ------------------------------------------------------------------- rows
ROWS = [(1, 1, 1, 1), (1, 8, 64, 2048), (3, 2, 4, 7), (5, 3, 4, 8), (16, 8, 64, 512), (33, 4, 9, 520), (7, 6, 17, 1337),
        (64, 5, 3, 1031), (9, 8, 8, 2056), (4, 2, 5, 4099), (130, 1, 6, 640), (3, 64, 80, 100), (2, 9, 3, 9000), (2000, 8, 64, 136)]


def some_order(dev, tokens, k, n, seed, away=0.2):
    g = gen(dev, seed)
    e = torch.randint(0, n, (tokens, k), generator=g, device=dev)
    e[torch.rand(tokens, k, generator=g, device=dev) < away] = -1
    if tokens > 2:
        e[1] = -1  # a token of no expert
    return mr.order_by_expert(e, n)


def kept(order):
    return order.place < order.offsets[-1]


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("tokens, k, n, width", ROWS)
def test_dispatch(dev, tokens, k, n, width, t):
    order = some_order(dev, tokens, k, n, width)
    x = randn(dev, 1, tokens, width).to(t)
    want = torch.zeros(tokens * k, width, dtype=t, device=dev)
    each = x[:, None].expand(-1, k, -1)
    want[order.place.long()[kept(order)]] = each[kept(order)]
    assert torch.equal(mr.dispatch_rows(x, order), want)
    for lay in (lambda v: strided(v, width + 24), lambda v: strided(v, width + 3), shifted):
        assert torch.equal(mr.dispatch_rows(lay(x), order), want)


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("tokens, k, n, width", ROWS)
def test_combine(dev, tokens, k, n, width, t):
    order = some_order(dev, tokens, k, n, width)
    y = randn(dev, 2, tokens * k, width).to(t)
    y[int(order.offsets[-1]):] = math.nan  # rows of no expert are not read
    w, r = torch.softmax(randn(dev, 3, tokens, k), 1), randn(dev, 4, tokens, width).to(t)
    rows = torch.where(kept(order)[:, :, None], y[order.place.long()].double(), 0.0)
    for weights, residual in ((w, r), (w, None), (None, r), (None, None)):
        part = rows if weights is None else rows * weights.double()[:, :, None]
        want, size = part.sum(1), part.abs().sum(1)
        if residual is not None:
            want, size = want + residual.double(), size + residual.double().abs()
        tol = want.abs() * H[t] * 1.01 + (k + 1) * U * size + TINY[t]
        within(mr.combine_rows(y, order, weights=weights, residual=residual), want, tol)
        for lay in (lambda v: strided(v, width + 3), shifted):
            within(mr.combine_rows(lay(y), order, weights=weights, residual=None if residual is None else lay(residual)), want, tol)
    assert torch.equal(mr.dispatch_rows_backward(y, order), mr.combine_rows(y, order))


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("tokens, k, n, width", ROWS)
def test_combine_backward(dev, tokens, k, n, width, t):
    order = some_order(dev, tokens, k, n, width)
    y, dout = randn(dev, 2, tokens * k, width).to(t), randn(dev, 5, tokens, width).to(t)
    y[int(order.offsets[-1]):] = math.nan
    w = torch.softmax(randn(dev, 3, tokens, k), 1)
    rows = torch.where(kept(order)[:, :, None], y[order.place.long()].double(), 0.0)
    dots = (rows * dout.double()[:, None]).sum(2)
    # a lane's terms, 6 additions across the wave, one for every 2048 columns (1024 of float32)
    d_tol = (rows * dout.double()[:, None]).abs().sum(2) * (width / 64 + 16 + 8 + width / 1024) * U
    for weights in (w, None):
        each = dout.double()[:, None].expand(-1, k, -1) * (1.0 if weights is None else weights.double()[:, :, None])
        want = torch.zeros(tokens * k, width, dtype=torch.float64, device=dev)
        want[order.place.long()[kept(order)]] = each[kept(order)]
        for lay in (lambda v: v, lambda v: strided(v, width + 3), shifted):
            drows, dweights = mr.combine_rows_backward(lay(dout), lay(y), order, weights)
            within(drows, want, want.abs() * (H[t] * 1.01 + U) + TINY[t], "drows")
            within(dweights, dots, d_tol, "dweights")


def test_places_that_are_no_rows_are_left_out(dev):
    """An order that is none (places out of range, offsets out of range) reads and writes inside the tensors only."""
    tokens, k, n, width = 6, 3, 4, 40
    order = some_order(dev, tokens, k, n, 1, away=0.0)
    place = order.place.clone()
    place[0, 1], place[2, 0], place[3, 2] = -1, tokens * k, 1 << 30
    for last in (tokens * k, 1 << 30, -5):
        offsets = order.offsets.clone()
        offsets[-1] = last
        bad = mr.ExpertOrder(offsets, place)
        ok = (place >= 0) & (place < min(max(last, 0), tokens * k))
        x, y, w = randn(dev, 1, tokens, width), randn(dev, 2, tokens * k, width), randn(dev, 3, tokens, k)
        out = mr.combine_rows(y, bad, weights=w)
        rows = torch.where(ok[:, :, None], y[place.clamp(0, tokens * k - 1).long()], 0.0).double()
        want = (rows * w.double()[:, :, None]).sum(1)
        within(out, want, 8 * U * (rows * w.double()[:, :, None]).abs().sum(1) + 1e-30)
        drows, dots = mr.combine_rows_backward(x, y, bad, w)
        assert bool((dots[~ok] == 0).all())
        got = mr.dispatch_rows(x, bad)
        at = place.long()[ok]
        assert torch.equal(got[at], x[:, None].expand(-1, k, -1)[ok])


def test_sorted_rows_past_four_gigabytes(dev):
    tokens, k, n, width = 40000, 8, 3, 8192  # 5.2e9 bytes of sorted bf16 rows
    e = torch.full((tokens, k), 1, dtype=torch.int32, device=dev)
    e[7, 3] = 2  # the last sorted row
    order = mr.order_by_expert(e, n)
    assert int(order.place[7, 3]) == tokens * k - 1
    x = randn(dev, 1, tokens, width).to(BF)
    rows = mr.dispatch_rows(x, order)
    assert torch.equal(rows[-1], x[7]) and torch.equal(rows[-2], x[-1]) and torch.equal(rows[: 8], x[:1].expand(8, -1))
    out = mr.combine_rows(rows, order)
    assert torch.equal(out[[0, 7, tokens - 1]], x[[0, 7, tokens - 1]] * 8)  # a power of two: exact
    w = torch.full((tokens, k), 0.5, device=dev)
    drows, dweights = mr.combine_rows_backward(x, rows, order, w)
    assert torch.equal(drows[-1], x[7] * 0.5)
    want = x[[0, 7, tokens - 1]].double().square().sum(1)
    within(dweights[[0, 7, tokens - 1]], want[:, None].expand(-1, k), want[:, None] * (width / 64 + 40) * U)


# ---------------------------------------------------------- run of them all
def block(x, wr, bank, k):
    """A token's experts and back, as a model runs it, with the gradients of everything."""
    n = bank.shape[0]
    logits = x.float() @ wr
    routed = mr.route_tokens(logits, k)
    order = mr.order_by_expert(routed.experts, n)
    rows = mr.dispatch_rows(x, order)
    y = mr.grouped_matmul(rows, bank, order.offsets)
    out = mr.combine_rows(y, order, weights=routed.weights, residual=x)
    dout = (out.float() * 0.01).to(x.dtype)
    dy, dweights = mr.combine_rows_backward(dout, y, order, routed.weights)
    dbank = mr.grouped_weight_grad(dy, rows, order.offsets)
    drows = mr.grouped_matmul(dy, bank, order.offsets, transpose=True)
    dx = mr.dispatch_rows_backward(drows, order)
    dlogits = mr.route_tokens_backward(dweights, logits, routed)
    return out, dbank, dx, dlogits, routed.weights, order.place


def test_the_run_captured_and_replayed(dev):
    tokens, width, n, k = 300, 256, 12, 3
    x, wr, bank = randn(dev, 1, tokens, width).to(BF), randn(dev, 2, width, n) / 16, (randn(dev, 3, n, width, width) / 16).to(BF)
    block(x, wr, bank, k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            block(x, wr, bank, k)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block(x, wr, bank, k)
    for seed in range(4):
        x.copy_(randn(dev, 10 + seed, tokens, width))
        graph.replay()
        want = block(x, wr, bank, k)
        torch.cuda.synchronize()
        for g, e in zip(got, want):
            assert torch.equal(g, e)


def test_the_run_against_formulas(dev):
    """Out of the run's gradients, those that go through every operator, in 64 bits from the stored 16-bit values."""
    tokens, width, n, k = 77, 128, 6, 2
    x, wr, bank = randn(dev, 1, tokens, width).to(BF), randn(dev, 2, width, n) / 16, (randn(dev, 3, n, width, width) / 11).to(BF)
    out, dbank, dx, dlogits, weights, _ = block(x, wr, bank, k)
    xd = x.double()
    l = xd @ wr.double()
    e = chosen_of(l, k)
    w = torch.softmax(l.gather(1, e), 1)
    y = torch.einsum("tjnk,tk->tjn", bank.double()[e], xd)
    y16 = y.to(BF).double()
    want = xd + (w[:, :, None] * y16).sum(1)
    # y's own rounding where it falls the other way, the logits' product in float32, the weights', the output's rounding
    size = xd.abs() + (w[:, :, None] * y16.abs()).sum(1)
    within(out, want, size * (2 * H[BF] + 300 * U), "out")
    dout = (out.float() * 0.01).to(BF).double()
    dw = (dout[:, None] * y16).sum(2)
    c = (w * dw).sum(1, keepdim=True)
    want = torch.zeros_like(l).scatter_add_(1, e, w * (dw - c))
    tol = torch.zeros_like(l).scatter_add_(1, e, w * ((dout[:, None] * y16).abs().sum(2) + ((dout[:, None] * y16).abs().sum(2) * w).sum(1, keepdim=True)))
    within(dlogits, want, tol * (2 * H[BF] + 300 * U) + 1e-30, "dlogits")
    assert bool((weights[:, 0] >= weights[:, 1]).all())


def test_another_stream(dev):
    tokens, width, n, k = 500, 640, 32, 4
    logits, x = randn(dev, 1, tokens, n), randn(dev, 2, tokens, width).to(BF)

    def all_of(**kw):
        r = mr.route_tokens(logits, k, **kw)
        o = mr.order_by_expert(r.experts, n, **kw)
        rows = mr.dispatch_rows(x, o, **kw)
        return [*r, *o, rows, mr.combine_rows(rows, o, weights=r.weights, residual=x, **kw),
                *mr.combine_rows_backward(x, rows, o, r.weights, **kw), mr.route_tokens_backward(r.weights, logits, r, **kw)]

    want = all_of()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = all_of(stream=s)
    s.synchronize()
    assert all(torch.equal(g, e) for g, e in zip(got, want))
