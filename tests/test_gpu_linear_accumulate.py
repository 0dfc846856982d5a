"""block_scaled_matmul into a 16-bit C that holds something: the float32 product
and C are added in float32 and rounded once, in every form of the product."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

E4 = torch.float8_e4m3fn
# few rows, 128 x 128 tiles, large tiles, split contractions, and sizes that are no whole 16-byte units
SIZES = [(5, 96, 384), (50, 77, 200), (300, 200, 256), (290, 130, 211), (4200, 4100, 192), (16, 64, 8192), (200, 120, 4096)]


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


def randn(dev, seed, *shape):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device=dev)


@pytest.mark.parametrize("t", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("b_square", [False, True])
@pytest.mark.parametrize("m, n, k", SIZES)
def test_one_rounding(dev, m, n, k, b_square, t):
    """C nearly cancels the product, so a rounding of the product alone would be most of what is left.  Operands between
    1 and 2 with 3 binary places: products have 6 and sums are below 2^14, exact in float32 and on 8-bit cores alike."""
    a, b = (1 + randn(dev, seed, rows, k).abs().remainder(1).mul(8).floor() / 8 for seed, rows in ((1, m), (2, n)))
    kb = (k + 127) // 128
    sa, sb = torch.ones(m, kb, device=dev), torch.ones((n + 127) // 128 if b_square else n, kb, device=dev)
    product = a.double() @ b.double().t().contiguous()
    # whole 16-byte units, rows of C that are none, rows of A and B that are none
    for pad, odd in ((0, 0), (3, 0), (0, 5)):
        x, y = (torch.zeros(v.shape[0], (k + 15) // 16 * 16 + odd, device=dev).to(E4)[:, :k] for v in (a, b))
        x.copy_(a)
        y.copy_(b)
        c = torch.zeros(m, n + pad, dtype=t, device=dev)[:, :n]
        c.copy_(-product)
        want = (product + c.double()).to(t)
        mr.block_scaled_matmul(x, sa, y, sb, out=c, accumulate=True)
        assert torch.equal(c, want), f"{int((c != want).sum())} of {c.numel()} off"


@pytest.mark.parametrize("m, n", [(8, 64), (300, 200), (4200, 4100)])
def test_a_product_past_the_range_of_fp16(dev, m, n):
    """65536 - 40000 = 25536 is an fp16 value; 65536 is none."""
    a, b = torch.full((m, 128), 16.0, device=dev).to(E4), torch.full((n, 128), 32.0, device=dev).to(E4)
    c = torch.full((m, n), -40000.0, device=dev, dtype=torch.float16)
    mr.block_scaled_matmul(a, torch.ones(m, 1, device=dev), b, torch.ones(n, 1, device=dev), out=c, accumulate=True)
    assert bool((c == 25536).all()), c.flatten()[:4]
