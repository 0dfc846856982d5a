"""The mean and the reciprocal deviation that layer norm stores, on the GPU."""

import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

from test_gpu_linear import BF, F32, HF, randn  # noqa: E402


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("width", [3, 500, 1337, 5000, 9000])
def test_rows_that_hold_no_numbers(dev, width, t):
    """As the formula has it: the deviation is NaN, and so are y and dx; other rows stay."""
    rows, nan, inf = 9, math.nan, math.inf
    w, b = 1 + 0.2 * randn(dev, 3, width), randn(dev, 4, width)
    x, dy = randn(dev, 1, rows, width).to(t), randn(dev, 2, rows, width).to(t)
    clean = mr.layer_norm_forward(x, w, b, 1e-5)
    clean_dx = mr.layer_norm_backward(dy, clean.h, clean.mean, clean.rstd, w)[0]
    x[1, width - 1], x[3, 0], x[5, width // 2], x[7, 0], x[7, width - 1], x[8, 1], x[8, 2] = nan, inf, -inf, inf, -inf, inf, inf
    out = mr.layer_norm_forward(x, w, b, 1e-5)
    bad = torch.tensor([0, 1, 0, 1, 0, 1, 0, 1, 1], dtype=torch.bool, device=dev)
    assert bool(out.rstd[bad].isnan().all()), out.rstd
    assert bool(out.y[bad].isnan().all())
    for g, e in zip(out[1:4], clean[1:4]):
        assert torch.equal(g[~bad], e[~bad])
    dx = mr.layer_norm_backward(dy, out.h, out.mean, out.rstd, w)[0]
    assert bool(dx[bad].isnan().all()) and torch.equal(dx[~bad], clean_dx[~bad])


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("width", [1, 3, 500, 1337, 5000, 9000])
def test_mean_of_rows_that_hold_infinity(dev, width, t):
    """Infinities of one sign: that infinity; of both, or with a NaN beside them: NaN."""
    inf = math.inf
    x = randn(dev, 1, 6, width).to(t)
    x[1, 0], x[3, width // 2], x[4, 0], x[5, width - 1] = inf, -inf, inf, math.nan
    x[4, width - 1] = -inf
    mean = mr.layer_norm_forward(x, torch.ones(width, device=dev), None, 1e-5).mean
    want = x.double().mean(1)
    assert bool((mean.isnan() == want.isnan()).all()) and bool((mean.isinf() == want.isinf()).all())
    assert mean[1] == inf and mean[3] == -inf and bool(torch.isfinite(mean[[0, 2]]).all())


def rows_of_exact_sums(rows, width):
    """Rows of eight-bit numbers times 256 below 2^16 in size, signs in turn, whose groups of eight columns add up to
    zero, but for column 7: one to 253, odd.  A row's sum is below 2^17, odd beside multiples of four, and no sum on the
    way to it, however the groups are joined, takes more than 24 bits."""
    g = torch.Generator().manual_seed(width)
    a = torch.randint(129, 255, (rows, width // 2), generator=g).double()
    step = torch.tensor([1.0, -1.0]).double().repeat(width // 4)
    x = torch.stack([a, -(a + step)], 2).view(rows, width) * 256
    x[:, 7] = torch.randint(0, 64, (rows,), generator=g).double() * 4 + 1
    return x


@pytest.mark.parametrize("t, width", [(BF, 1024), (BF, 2048), (BF, 4096), (BF, 8192), (BF, 16384), (HF, 1024), (HF, 2048), (HF, 4096)])
def test_mean_of_16_bit_rows(dev, width, t):
    """The exact mean, a float32, comes out as it is.  Differences of the row's values from a number of the row's own
    type are multiples of its last place: 2^17 over 2^-6 (bf16, 16384 columns: means from two on) or over 2^-7 (fp16,
    4096 columns: from eight on) is 2^24 at most, so they and their sums are exact.  Differences from a float32 mean
    take up to 2^16 over 2^-10 and would all be rounded the same way, by 2^-10."""
    x = rows_of_exact_sums(40, width)
    want = x.mean(1)
    assert torch.equal(want.float().double(), want) and torch.equal(x.to(t).double(), x)
    out = mr.layer_norm_forward(x.to(t).to(dev), torch.ones(width, device=dev), None, 1e-5)
    got = out.mean.cpu().double()
    assert torch.equal(got, want), float((got - want).abs().max())


@pytest.mark.parametrize("width", [100, 1337, 5000])
def test_rows_beyond_the_range_of_sums(dev, width):
    """A sum that overflows: as a row with infinity; squares that do: a deviation's reciprocal of 0."""
    x = torch.full((3, width), 3e38, device=dev)
    x[1], x[2] = 1.0, 1e21
    x[2, ::2] = -1e21
    out = mr.layer_norm_forward(x, torch.ones(width, device=dev), None, 1e-5)
    assert out.mean[0] == math.inf and bool(out.rstd[0].isnan()) and bool(out.y[0].isnan().all())
    assert out.mean[1] == 1 and bool((out.y[1] == 0).all())
    assert out.rstd[2] == 0 and bool((out.y[2] == 0).all())
