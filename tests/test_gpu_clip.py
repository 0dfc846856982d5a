"""Gradient clipping on the GPU against 64-bit formulas.

Squares and sums are float64: n terms, however added up, are off by at most n
2^-53 of their sum, and no chain of additions here is longer than 1 / 64 of a
gradient's values and 200 more.  A scaled value is off by the float64 product, by half a
step of float32 and half a step of its type, H[t] = finfo(t).eps / 2."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

from test_gpu_linear import BF, F32, H, HF, TINY, U, randn, within  # noqa: E402


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


def norms_of(grads):
    each = torch.stack([g.double().square().sum() for g in grads])
    return float(each.sum().sqrt()), each.sqrt()


def check(grads, max_norm, outs=None):
    n, each = norms_of(grads)
    before = [g.double() for g in grads]
    got, norms = mr.clip_gradients_batched(grads, max_norm, outs=outs, return_norms=True)
    assert got.dtype == norms.dtype == torch.float64 and got.dim() == 0
    rel = (max(g.numel() for g in grads) / 64 + 200) * 2.0 ** -53
    assert abs(float(got) - n) <= n * rel * 2
    within(norms, each, each * rel * 2 + 1e-300, "norms")
    by = max_norm / n if n > max_norm else 1.0
    for g, b, o in zip(grads, before, outs or grads):
        if by == 1.0:
            assert torch.equal(o, g) if o.dtype == g.dtype else torch.equal(o, g.to(o.dtype))
        else:
            want = b * by
            within(o, want, want.abs() * (H[o.dtype] * 1.01 + U + 2 * rel) + TINY[o.dtype])
        if outs is not None:
            assert torch.equal(g.double(), b)


SETS = [[(1,)], [(3,), (64, 128), (64, 128)], [(1000, 1000)], [(7, 11), (5,), (1, 1), (2049,), (130, 257)],
        [(17 * i + 1, 3 * i + 1) for i in range(120)], [(4, 33, 65), (2, 3, 4, 5), ()], [(16384 * 40 + 5,), (8,)]]


@pytest.mark.parametrize("t", [F32, BF, HF])
@pytest.mark.parametrize("shapes", SETS)
def test_clip(dev, shapes, t):
    def make():
        return [randn(dev, i, *(s or (1,))).to(t).reshape(s) for i, s in enumerate(shapes)]

    n, _ = norms_of(make())
    check(make(), 0.31 * n)
    check(make(), 1.5 * n)
    check(make(), math.inf)
    for to in {t, F32}:
        check(make(), 0.31 * n, [torch.empty(s, dtype=to, device=dev) for s in shapes])
        check(make(), 1.5 * n, [torch.empty(s, dtype=to, device=dev) for s in shapes])


def test_types_together(dev):
    grads = [randn(dev, 1, 100, 30), randn(dev, 2, 777).to(BF), randn(dev, 3, 5, 6, 7).to(HF)]
    check(grads, 3.0, [torch.empty(g.shape, device=dev) for g in grads])
    check(grads, 3.0)


def test_where_gradients_lie(dev):
    """Views of larger tensors, transposed ones, odd addresses: the values around them stay."""
    for t in (F32, BF):
        big = torch.full((40, 300), 7.0, dtype=t, device=dev)
        views = [big[1:20, 3:100], big[31:, :], big[21:30, 101:299].t(), big[30, 1:2]]
        for i, v in enumerate(views):
            v.copy_(randn(dev, i, *v.shape))
        mask = torch.ones_like(big, dtype=torch.bool)
        for v in views:
            mask.as_strided(v.shape, v.stride(), v.storage_offset()).fill_(False)
        check(views, 2.0)
        assert bool((big[mask] == 7).all())
        with pytest.raises(B.MatrixRootsError):  # interleaved columns: the bytes from first to last overlap
            mr.clip_gradients_batched([big[:, :100], big[:, 100:]], 2.0)
        outs = [torch.empty(60, 100, device=dev)[2:21, :97], torch.empty(9, 304, device=dev)[:, :300]]
        check(views[:2], 1.0, outs)
    flat = torch.zeros(10001, dtype=BF, device=dev)
    flat[1:].copy_(randn(dev, 5, 10000))
    check([flat[1:]], 1.0)
    check([flat[1:]], 0.5, [torch.zeros(10003, device=dev)[3:]])


def test_many(dev):
    """More gradients than a launch takes, dense and in rows, and more partial sums than a workgroup adds up by itself."""
    flat = torch.zeros(4300 * 7, device=dev)
    flat.copy_(randn(dev, 1, 4300 * 7))
    big = randn(dev, 2, 130 * 20, 40).to(BF)
    rows = [big[20 * i:20 * i + 9, 3:30] for i in range(130)]
    check([flat[7 * i:7 * i + 1 + i % 7] for i in range(4300)], 3.0)
    check(rows, 3.0)
    check(rows + [flat[7 * i:7 * i + 5] for i in range(4300)], 1.0)
    check(rows, 0.7, [torch.empty(9, 31, device=dev)[:, :27] for _ in rows])


def test_empty_and_zero(dev):
    zero = torch.zeros(50, 3, device=dev)
    check([zero], 0.0)
    check([zero, torch.zeros(0, 4, device=dev), randn(dev, 1, 9)], 0.5)
    got = [randn(dev, 1, 9)]
    mr.clip_gradients_batched(got, 0.0)
    assert bool((got[0] == 0).all())


def test_squares_out_of_float32s_range(dev):
    check([torch.full((300,), 1e30, device=dev)], 1e20)
    check([torch.full((300,), 1e-30, device=dev)], 1e-32)
    check([torch.full((300,), 1e-42, device=dev)], 1e30)  # no normal numbers


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_norms_that_are_not_finite(dev, bad):
    """The gradients stay as they are, copies too; the norm says so."""
    grads = [randn(dev, 1, 500), randn(dev, 2, 70, 70)]
    grads[1][3, 4] = bad
    before = [g.clone() for g in grads]
    outs = [torch.empty_like(g) for g in grads]
    for o in (None, outs):
        n, norms = mr.clip_gradients_batched(grads, 1.0, outs=o, return_norms=True)
        assert not math.isfinite(float(n)) and math.isnan(float(n)) == math.isnan(bad)
        assert math.isfinite(float(norms[0])) and not math.isfinite(float(norms[1]))
        for g, b in zip(o or grads, before):
            assert torch.equal(g.view(torch.int32), b.view(torch.int32))


def test_more_than_four_gigabytes(dev):
    g = torch.zeros(5, 1 << 28, dtype=BF, device=dev)  # 1.3e9 values, 2.7e9 bytes
    o = torch.empty(5, 1 << 28, device=dev)  # 5.4e9 bytes
    g[4, -1], g[0, 0] = 3.0, 4.0
    n = mr.clip_gradients_batched([g], 1.0, outs=[o])
    assert float(n) == 5.0
    assert abs(float(o[4, -1]) - 0.6) <= 0.6 * U and abs(float(o[0, 0]) - 0.8) <= 0.8 * U and int((o != 0).sum()) == 2


def test_another_stream_and_two_captured_calls(dev):
    """Two graphs of calls, replayed in turn and on other gradients, give what eager calls give."""
    a, b = [randn(dev, i, 300, 70) for i in range(3)], [randn(dev, i, 900) for i in range(60)]
    outs = [torch.empty_like(g) for g in a], [torch.empty_like(g) for g in b]

    def one(i, **k):
        return mr.clip_gradients_batched((a, b)[i], 1.0 + i, outs=outs[i], return_norms=True, **k)

    s = torch.cuda.Stream()
    want = one(0)
    want_out = [o.clone() for o in outs[0]]
    s.wait_stream(torch.cuda.current_stream())
    got = one(0, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and all(torch.equal(o, w) for o, w in zip(outs[0], want_out))
    graphs, kept = [], []
    for i in range(2):
        one(i)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept.append(one(i))
        graphs.append(graph)
    for seed in range(3):
        for j, g in enumerate(a + b):
            g.copy_(randn(dev, 100 * seed + j, *g.shape) * (seed + 0.5))
        for i in (0, 1):
            graphs[i].replay()
        torch.cuda.synchronize()
        got = [[kept[i][0].clone(), kept[i][1].clone()] + [o.clone() for o in outs[i]] for i in (0, 1)]
        for i in (0, 1):
            n = one(i)
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(got[i], [*n, *outs[i]]))
