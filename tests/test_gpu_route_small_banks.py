"""Routing among a few dozen experts: many of a token's logits reach the k-th of the
lanes' largest there, or fewer lanes than k hold any."""

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from matrix_roots_amd import binding as B  # noqa: E402

from test_gpu_experts import check_route  # noqa: E402
from test_gpu_linear import BF, F32, gen, randn  # noqa: E402


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("experts", [9, 16, 20, 25, 28, 29, 32, 33, 36, 40, 48, 63, 100, 128])
@pytest.mark.parametrize("k", [5, 7, 8])
def test_route(dev, experts, k):
    logits = randn(dev, experts, 700, experts)
    logits[600:] = torch.randint(-1, 2, (100, experts), generator=gen(dev, k), device=dev).float()
    logits[650:, ::3] = -float("inf")
    for t in (F32, BF):
        for normalize in (True, False):
            check_route(logits.to(t), k, normalize)
