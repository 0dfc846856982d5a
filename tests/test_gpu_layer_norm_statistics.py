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
