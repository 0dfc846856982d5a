"""The operators around a bank of experts on a stream that has no order with the
current one: a block freed while a copy out of it still waits on the current stream
is not written by a result of its size."""

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
    order = mr.order_by_expert(torch.randint(0, 5, (ROWS, 1), generator=g, device=dev), 5)
    n = mr.layer_norm_forward(x, w, w, 1e-5)
    share = torch.rand(ROWS, 1, generator=g, device=dev)
    # (operator, its result of ROWS x WIDTH 16-bit values)
    return {
        "norm": lambda **k: mr.layer_norm_forward(x, w, w, 1e-5, **k).y,
        "norm_grad": lambda **k: mr.layer_norm_backward(x, n.h, n.mean, n.rstd, w, **k)[0],
        "dispatch": lambda **k: mr.dispatch_rows(x, order, **k),
        "combine": lambda **k: mr.combine_rows(x, order, weights=share, **k),
        "combine_grad": lambda **k: mr.combine_rows_backward(x, n.y, order, share, **k)[0],
    }


@pytest.mark.parametrize("name", ["norm", "norm_grad", "dispatch", "combine", "combine_grad"])
def test_memory_that_the_current_stream_still_reads_is_not_written(dev, name):
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


def test_clipping_in_place_on_another_stream(dev):
    """Ordered with the current stream by the caller; the norm comes from the call's stream and is read on the current one."""
    grads = [torch.full((1000, 1000), 0.5, device=dev), torch.full((77,), 2.0, dtype=BF, device=dev)]
    want = (250000.0 + 308.0) ** 0.5
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    n = mr.clip_gradients_batched(grads, 5.0, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert abs(float(n) - want) < 1e-9
    # half a step of float32; of bf16, 2^-8, and of the float32 before it
    assert abs(float(grads[0][0, 0]) - 2.5 / want) < 2.0 ** -24 * 0.01
    assert abs(float(grads[1][5]) - 10 / want) < (2.0 ** -8 + 2.0 ** -23) * 10 / want
