"""The linear-layer operators on a stream that has no order with the current one."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

BF = torch.bfloat16
ROWS, WIDTH = 4096, 2048


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


def calls(dev):
    g = torch.Generator(device=dev)
    g.manual_seed(1)
    x = torch.randn(ROWS, WIDTH, generator=g, device=dev).to(BF)
    w = torch.ones(WIDTH, device=dev)
    bank = torch.randn(1, WIDTH, WIDTH, generator=g, device=dev).to(BF)
    off = torch.tensor([0, ROWS], dtype=torch.int32, device=dev)
    q = mr.quantize_blocks(x)
    b = mr.quantize_blocks(bank[0], block="square")
    n = mr.rms_norm_forward(x, w, 1e-6)
    # (operator, its result of ROWS x WIDTH 16-bit values)
    return {
        "norm": lambda **k: mr.rms_norm_forward(x, w, 1e-6, **k).y,
        "norm_grad": lambda **k: mr.rms_norm_backward(x, n.h, n.rstd, w, **k)[0],
        "matmul": lambda **k: mr.block_scaled_matmul(q.q, q.scales, b.q, b.scales, **k),
        "grouped": lambda **k: mr.grouped_matmul(x, bank, off, **k),
    }


@pytest.mark.parametrize("name", ["norm", "norm_grad", "matmul", "grouped"])
def test_memory_that_the_current_stream_still_reads_is_not_written(dev, name):
    """A block freed while a copy out of it waits on the current stream: a result of its size goes elsewhere."""
    call = calls(dev)[name]
    want = call()
    s = torch.cuda.Stream()
    big = torch.ones(8192, 8192, device=dev)
    held, late = torch.full((ROWS, WIDTH), 3.0, dtype=BF, device=dev), torch.empty(ROWS, WIDTH, dtype=BF, device=dev)
    torch.cuda.synchronize()
    for _ in range(4):
        big = big @ big * 1e-4  # tens of milliseconds
    late.copy_(held)
    del held
    got = call(stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert bool((late == 3).all())
    assert torch.equal(got, want)


def test_results_are_not_reused_while_the_current_stream_reads_them(dev):
    """The other way round: a result freed while a copy out of it waits on the current stream."""
    call = calls(dev)["norm"]
    want = call()
    s = torch.cuda.Stream()
    big, late = torch.ones(8192, 8192, device=dev), torch.empty(ROWS, WIDTH, dtype=BF, device=dev)
    x = torch.zeros(ROWS, WIDTH, dtype=BF, device=dev)
    torch.cuda.synchronize()
    got = call(stream=s)
    s.synchronize()
    for _ in range(4):
        big = big @ big * 1e-4
    late.copy_(got)
    del got
    other = mr.rms_norm_forward(x, torch.ones(WIDTH, device=dev), 1e-6, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(late, want) and bool((other.y == 0).all())
