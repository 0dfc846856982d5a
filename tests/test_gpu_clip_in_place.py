"""Gradients clipped in place against copies taken before the call, and against the
same call into outputs: what a training step calls it for."""

import ctypes
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

from test_gpu_clip import SETS, norms_of  # noqa: E402
from test_gpu_linear import BF, F32, H, HF, TINY, U, randn, within  # noqa: E402


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


def bits(t):
    return t.contiguous().view(torch.int32 if t.dtype == F32 else torch.int16)


@pytest.mark.parametrize("t", [F32, BF, HF])
@pytest.mark.parametrize("shapes", SETS)
def test_values_below_the_limit_stay(dev, shapes, t):
    """Bit for bit, zeros' signs among them; in place and as copies of the same type, copies in float32 by value."""
    grads = [randn(dev, i, *(s or (1,))).to(t).reshape(s) for i, s in enumerate(shapes)]
    grads[0].view(-1)[0] = -0.0
    before = [g.clone() for g in grads]
    n, _ = norms_of(grads)
    for limit in (1.5 * n + 1e-30, math.inf):
        got = mr.clip_gradients_batched(grads, limit)
        assert abs(float(got) - n) <= n * 1e-9
        assert all(torch.equal(bits(g), bits(b)) for g, b in zip(grads, before))
        for to in (t, F32):
            outs = [torch.full(s, 7.0, dtype=to, device=dev) for s in shapes]
            mr.clip_gradients_batched(grads, limit, outs=outs)
            assert all(torch.equal(bits(o), bits(b.to(to))) for o, b in zip(outs, before))
            assert all(torch.equal(bits(g), bits(b)) for g, b in zip(grads, before))


@pytest.mark.parametrize("t", [F32, BF, HF])
@pytest.mark.parametrize("shapes", SETS)
def test_values_above_the_limit_are_scaled(dev, shapes, t):
    """In place as into outputs of the type, and as the formula has it: the product's half step, a step of float32, the
    norm's (its sum has at most a 64th of the values and 200 more terms one after another, 2^-53 each)."""
    grads = [randn(dev, i, *(s or (1,))).to(t).reshape(s) for i, s in enumerate(shapes)]
    before = [g.double() for g in grads]
    n, _ = norms_of(grads)
    outs = [torch.full(s, 7.0, dtype=t, device=dev) for s in shapes]
    mr.clip_gradients_batched(grads, 0.31 * n, outs=outs)
    assert all(torch.equal(g.double(), b) for g, b in zip(grads, before))
    mr.clip_gradients_batched(grads, 0.31 * n)
    rel = (max(g.numel() for g in grads) / 64 + 200) * 2.0 ** -52
    for g, o, b in zip(grads, outs, before):
        assert torch.equal(bits(g), bits(o))
        want = b * 0.31
        within(g, want, want.abs() * (H[t] * 1.01 + U + rel) + TINY[t])


def test_no_gradients(dev):
    """The C entry point without any: the norm is 0."""
    lib = B.library()
    norms = torch.full((1,), 7.0, dtype=torch.float64, device=dev)
    assert lib.clip_gradients_batched_workspace(None, 0) == 0
    assert lib.clip_gradients_batched(None, 0, 1.0, norms.data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream) == 0
    assert float(norms[0]) == 0.0
    # gradients without values: a norm each
    probs = (B.ClipProblem * 3)(B.ClipProblem(0, 5, 0, 0, 0, 0, B.MR_F32, B.MR_F32), B.ClipProblem(5, 0, 0, 0, 0, 0, B.MR_BF16, B.MR_BF16),
                                B.ClipProblem(7, 0, 0, 3, 0, 0, B.MR_F16, B.MR_F16))
    at = ctypes.addressof(probs)
    norms = torch.full((4,), 7.0, dtype=torch.float64, device=dev)
    need = lib.clip_gradients_batched_workspace(at, 3)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    assert lib.clip_gradients_batched(at, 3, 1.0, norms.data_ptr(), ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream) == 0
    assert norms.tolist() == [0.0] * 4


@pytest.mark.parametrize("t", [F32, BF])
def test_columns(dev, t):
    """Columns of a matrix, in place and into outputs: the values around them stay."""
    big = torch.full((700, 9), 3.0, dtype=t, device=dev)
    kept = torch.full((41, 5, 3), 3.0, dtype=t, device=dev)
    grads = [big[:, 4:5], kept[:, :, 1:2]]
    for i, g in enumerate(grads):
        g.copy_(randn(dev, i, *g.shape))
    before = [g.double() for g in grads]
    n = float(sum(b.square().sum() for b in before).sqrt())
    rel = 300 * 2.0 ** -52
    for into in ([torch.zeros(700, 1, device=dev)], None):
        part = grads[:1] if into is not None else grads
        limit = 0.5 * (float(before[0].square().sum().sqrt()) if into is not None else n)
        norm = float(mr.clip_gradients_batched(part, limit, outs=into))
        assert abs(norm - 2 * limit) <= norm * rel
        for g, b in zip(into or part, before):
            within(g, b * 0.5, b.abs() * 0.5 * (H[g.dtype] * 1.01 + U + 2 * rel) + TINY[g.dtype])
    assert bool((big[:, :4] == 3).all()) and bool((big[:, 5:] == 3).all())
    assert bool((kept[:, :, 0] == 3).all()) and bool((kept[:, :, 2] == 3).all())
