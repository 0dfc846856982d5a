"""How often and in what order the linear-layer operators round, at values where it shows.

The 8-bit values of a block are its float32 values divided by the block's scale,
the quotient rounded to float32 and then to 8 bits, as a division in float32
gives them: compared bit for bit."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EIGHT = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


def randn(dev, seed, *shape):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=dev)


def divided(y, eight, tall):
    """(bytes, scales) of float32 y (on the CPU, whose division and conversion round to nearest even) for blocks of tall x 128."""
    dtype, top = EIGHT[eight]
    y = y.cpu()
    m, n = y.shape
    full = torch.zeros((m + tall - 1) // tall * tall, (n + 127) // 128 * 128)
    full[:m, :n] = y
    tiles = full.view(full.shape[0] // tall, tall, full.shape[1] // 128, 128)
    s = tiles.abs().amax((1, 3)).clamp_min(2.0 ** -100) / top
    return (tiles / s[:, None, :, None]).view(full.shape)[:m, :n].to(dtype).view(torch.uint8), s


def raw(q):
    return q.cpu().contiguous().view(torch.uint8)


@pytest.mark.parametrize("eight", ["e4m3", "e5m2"])
@pytest.mark.parametrize("block", ["vector", "square"])
@pytest.mark.parametrize("t", [BF, HF, F32])
def test_quantised_values_are_quotients(dev, t, block, eight):
    """Values of 8 significant bits meet the middle between two 8-bit values often; blocks of very large and very small
    values among them, and in float32 some of full length."""
    x = randn(dev, 1, 517, 392)
    x[:, 128:256] *= 1e30 if t != HF else 1e3
    x[128:256] *= 1e-25 if t != HF else 1e-2
    x = x.to(t)
    if t == F32:
        x[:400] = x[:400].to(BF).float()
    got = mr.quantize_blocks(x, eight, block=block, order="both")
    tall = 128 if block == "square" else 1
    for q, s, y in ((got.q, got.scales, x.float()), (got.qt, got.scales_t, x.float().t())):
        want, scales = divided(y, eight, tall)
        assert torch.equal(s.cpu(), scales)
        off = int((raw(q) != want).sum())
        assert off == 0, f"{off} of {want.numel()} values"


@pytest.mark.parametrize("eight", ["e4m3", "e5m2"])
@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows, width", [(70, 1024), (30, 2500), (4, 9001)])
def test_norm_quantises_quotients(dev, rows, width, t, eight):
    """Rows of 1 and -1 under eps 0 have rstd 1, so y is the weight with their signs: 8 significant bits, exact in both types."""
    x = torch.where(randn(dev, 2, rows, width) < 0, -1.0, 1.0).to(t)
    w = randn(dev, 3, width).to(BF).float()
    got = mr.rms_norm_forward(x, w, 0.0, eight=eight)
    assert bool((got.rstd == 1).all()) and torch.equal(got.y.float(), x.float() * w)
    want, scales = divided(got.y.float(), eight, 1)
    assert torch.equal(got.scales.cpu(), scales)
    off = int((raw(got.q) != want).sum())
    assert off == 0, f"{off} of {want.numel()} values"


@pytest.mark.parametrize("eight", ["e4m3", "e5m2"])
def test_norm_quantises_the_float32_values(dev, eight):
    got = mr.rms_norm_forward(randn(dev, 4, 300, 2500), 1 + 0.2 * randn(dev, 5, 2500), 1e-6, eight=eight)
    want, scales = divided(got.y, eight, 1)
    assert torch.equal(got.scales.cpu(), scales) and torch.equal(raw(got.q), want)
