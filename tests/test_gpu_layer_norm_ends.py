"""Ragged ends of layer norm's rows on the GPU: columns that two lanes hold."""

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
@pytest.mark.parametrize("width", [520, 1000, 1030, 1543, 2047, 2050, 4095, 4100, 6001, 6145, 8190, 8200, 12287, 12289, 16381])
def test_equal_columns_come_out_equal(dev, width, t):
    """Whichever lane and part of a row holds them: the columns that two lanes hold are stored by both."""
    rows = 60

    def spread(seed, *shape):
        v = randn(dev, seed, *shape)
        return v[..., torch.arange(width, device=dev) % 512].contiguous()

    x, r, dy = (spread(s, rows, 512).mul_(3).add_(1).to(t) for s in (1, 2, 3))
    w, b = 1 + 0.2 * spread(4, 512), spread(5, 512)
    for res in (r, None):
        out = mr.layer_norm_forward(x, w, b, 1e-5, residual=res)
        dx, dweight, dbias = mr.layer_norm_backward(dy, out.h, out.mean, out.rstd, w, dresidual=res)
        for name, v in (("h", out.h), ("y", out.y), ("dx", dx), ("dweight", dweight), ("dbias", dbias)):
            assert torch.equal(v[..., 512:], v[..., : width - 512]), name
