"""Scales of block_scaled_matmul whose product is no normal float32: every form of the
product multiplies a block's sum by A's scale and then by B's, so that what is finite
on the way stays what the formula says."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

U = 2.0 ** -24
H = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E4, E5 = torch.float8_e4m3fn, torch.float8_e5m2
# few rows, 128 x 128 tiles, large tiles (one chunk; several, the last one ragged), a split contraction of few and of more rows
SIZES = [(8, 300, 256), (300, 264, 384), (4200, 4100, 128), (4200, 4100, 400), (16, 64, 8192), (130, 100, 4096)]


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


def rows_at(x, aligned):
    """x in rows of whole 16-byte units, or one byte past them."""
    if aligned:
        return x
    flat = torch.zeros(x.numel() + 1, dtype=x.dtype, device=x.device)
    flat[1:] = x.reshape(-1)
    return flat[1:].view(x.shape)


def scales(dev, rows, k, square, value):
    return torch.full(((rows + 127) // 128 if square else rows, (k + 127) // 128), value, device=dev)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b_square", [False, True])
@pytest.mark.parametrize("a8", [E4, E5])
@pytest.mark.parametrize("m, n, k", SIZES)
def test_zero_sums_stay_zero_under_large_scales(dev, m, n, k, a8, b_square, out):
    """2^80 2^60 is past float32's range; a sum of zero is zero all the same, and one of 2^-18 is 2^122."""
    a, b = torch.zeros(m, k, device=dev), torch.zeros(n, k, device=dev)
    a[::2, 5], b[:, 5] = 2.0 ** -9, 2.0 ** -9  # one product of 2^-18
    a, b = a.to(a8), b.to(E4)
    want = torch.zeros(m, n, device=dev)
    want[::2] = 2.0 ** 122
    for aligned in (True, False):
        got = mr.block_scaled_matmul(rows_at(a, aligned), scales(dev, m, k, False, 2.0 ** 80), rows_at(b, aligned),
                                     scales(dev, n, k, b_square, 2.0 ** 60), out_dtype=out)
        assert torch.equal(got.float(), want), (aligned, got.float().isnan().sum())


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b_square", [False, True])
@pytest.mark.parametrize("a8", [E4, E5])
@pytest.mark.parametrize("m, n, k", SIZES)
def test_large_sums_keep_their_places_under_small_scales(dev, m, n, k, a8, b_square, out):
    """1.1 2^-70 1.7 2^-68 lies among float32's subnormal numbers, the results (2^23 of it a block) do not."""
    u, v = 1.1 * 2.0 ** -70, 1.7 * 2.0 ** -68
    a, b = torch.full((m, k), 256.0, device=dev).to(a8), torch.full((n, k), 256.0, device=dev).to(E4)
    sa, sb = scales(dev, m, k, False, u), scales(dev, n, k, b_square, v)
    want = k * 65536.0 * float(sa.flatten()[0].double()) * float(sb.flatten()[0].double())
    assert 2.0 ** -126 < want
    # the sum of a block is exact; two multiplications, k / 128 additions (and up to 16 parts), the output's rounding
    tol = want * ((2 + k / 128 + 16) * U + H[out])
    for aligned in (True, False):
        got = mr.block_scaled_matmul(rows_at(a, aligned), sa, rows_at(b, aligned), sb, out_dtype=out)
        worst = float((got.double() - want).abs().max())
        assert worst <= tol, (aligned, worst / want)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("b_square", [False, True])
@pytest.mark.parametrize("m, n, k", SIZES)
def test_rows_under_such_scales_keep_to_themselves(dev, m, n, k, b_square, out):
    """Every third row of A has scales whose product with B's is no normal number, in some blocks: small, small on
    zeros, zero, NaN.  The other rows keep their bits, these have the formula's values.  (Operands between 1 and 2 in
    magnitude with 3 binary places: the sums of a block are exact.)"""
    g = torch.Generator(device=dev)
    g.manual_seed(m + n + k)
    values, b = (torch.randn(r, k, generator=g, device=dev) for r in (m, n))
    values, b = (v.sign() * (1 + v.abs().remainder(1).mul(8).floor() / 8) for v in (values, b))
    b = b.to(E4)
    kb = (k + 127) // 128
    sa = torch.rand(m, kb, generator=g, device=dev) + 0.5
    sb = (torch.rand((n + 127) // 128 if b_square else n, kb, generator=g, device=dev) + 0.5) * 2.0 ** -60
    base = mr.block_scaled_matmul(values.to(E4), sa, b, sb, out_dtype=out)
    rows = torch.arange(m, device=dev)
    sa = sa.clone()
    small, zeros, zero, nan = (rows % 15 == 3 * i for i in range(4))
    sa[small, 0] = 1.3 * 2.0 ** -75  # 2^-135: the other blocks, where there are any, hold more
    values[small, 128:] = 0
    sa[zeros, -1] = 2.0 ** -109
    values[zeros, (kb - 1) * 128:] = 0
    sa[zero, 0] = 0
    sa[nan, kb // 2] = float("nan")
    a = values.to(E4)
    x = a.double() * sa.double().repeat_interleave(128, 1)[:, :k]
    s2 = sb.double().repeat_interleave(128, 1)[:, :k]
    y = b.double() * (s2.repeat_interleave(128, 0)[:n] if b_square else s2)
    want, mag = x.nan_to_num() @ y.t().contiguous(), x.nan_to_num().abs() @ y.abs().t().contiguous()
    # three factors of a block, the blocks' additions and up to 16 parts
    tol = mag * (3 + kb + 16) * U + want.abs() * H[out] * 1.01 + 2.0 ** -126 * H[out]
    touched = small | zeros | zero | nan
    for aligned in (True, False):
        got = mr.block_scaled_matmul(rows_at(a, aligned), sa, rows_at(b, aligned), sb, out_dtype=out)
        assert torch.equal(got[~touched], base[~touched])
        assert bool(got[nan].isnan().all())
        off = ~((got.double() - want).abs() <= tol) & ~nan[:, None]
        assert not bool(off.any()), (aligned, rows[off.any(1)][:5].tolist())
