"""block_scaled_matmul into a 16-bit C that holds something: the float32 product
and C are added in float32 and rounded once, in every form of the product."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

U = 2.0 ** -24
H = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
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
    """C nearly cancels the product, so a rounding of the product alone would be most of what is left."""
    a = mr.quantize_blocks(randn(dev, 1, m, k).abs())
    b = mr.quantize_blocks(randn(dev, 2, n, k).abs(), block="square" if b_square else "vector")
    x = a.q.double() * a.scales.double().repeat_interleave(128, 1)[:, :k]
    sb = b.scales.double().repeat_interleave(128, 1)[:, :k]
    y = b.q.double() * (sb.repeat_interleave(128, 0)[:n] if b_square else sb)
    product = x @ y.t().contiguous()  # its terms are positive: their magnitudes' sum too
    for pad in (0, 3):  # rows of C in whole 16-byte units or not
        c = torch.zeros(m, n + pad, dtype=t, device=dev)[:, :n]
        c.copy_(-product)
        want = product + c.double()
        mr.block_scaled_matmul(a.q, a.scales, b.q, b.scales, out=c, accumulate=True)
        # eight products together keep 17 bits below the largest: 8 2^-17 of the sum; then float32 sums, one rounding to t
        tol = product * (2.0 ** -14 + (2 * 128 + (k + 127) // 128 + 19) * U) + want.abs() * H[t] * 1.01 + TINY[t]
        off = (c.double() - want).abs() > tol
        assert not bool(off.any()), f"{int(off.sum())} of {off.numel()} off, worst {float(((c.double() - want).abs() / tol).max()):.3g} x tolerance"


@pytest.mark.parametrize("m, n", [(8, 64), (300, 200), (4200, 4100)])
def test_a_product_past_the_range_of_fp16(dev, m, n):
    """65536 - 40000 = 25536 is an fp16 value; 65536 is none."""
    a, b = torch.full((m, 128), 16.0, device=dev).to(E4), torch.full((n, 128), 32.0, device=dev).to(E4)
    c = torch.full((m, n), -40000.0, device=dev, dtype=torch.float16)
    mr.block_scaled_matmul(a, torch.ones(m, 1, device=dev), b, torch.ones(n, 1, device=dev), out=c, accumulate=True)
    assert bool((c == 25536).all()), c.flatten()[:4]
