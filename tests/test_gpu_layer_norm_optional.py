"""Layer norm on the GPU without its optional arguments: no bias, no mean or reciprocal
deviation stored, one of the parameters' gradients alone."""

import ctypes

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

import matrix_roots_amd as mr  # noqa: E402
from matrix_roots_amd import binding as B  # noqa: E402

from test_gpu_layer_norm import grad_reference, reference  # noqa: E402
from test_gpu_linear import BF, F32, H, HF, TINY, check_eight, randn, within  # noqa: E402

CODES = {F32: B.MR_F32, HF: B.MR_F16, BF: B.MR_BF16}


@pytest.fixture(scope="module")
def dev(gpu_available):
    B.library()
    return torch.device("cuda:0")


@pytest.mark.parametrize("t", [BF, HF, F32])
@pytest.mark.parametrize("rows, width", [(3, 5), (9, 1337), (33, 520), (65, 1000), (4, 2048), (2, 9000)])
def test_without_a_bias(dev, rows, width, t):
    x = (randn(dev, 1, rows, width).mul_(3) + 2 * randn(dev, 11, rows, 1)).to(t)
    w = 1 + 0.2 * randn(dev, 3, width)
    for w_, eight, keep in ((w, "e4m3", True), (w.to(t), "e5m2", True), (w, None, True), (w, "e4m3", False)):
        out = mr.layer_norm_forward(x, w_, None, 1e-5, keep_y=keep, eight=eight)
        mean, m_tol, rstd, r_tol, y, y_tol = reference(x, w_, None, 1e-5)
        within(out.mean, mean, m_tol + TINY[F32], "mean")
        within(out.rstd, rstd, r_tol, "rstd")
        if keep:
            within(out.y, y, y.abs() * H[t] * 1.01 + y_tol + TINY[t], "y")
        else:
            assert out.y is None
        if eight:
            check_eight(out.q, out.scales, y, eight, False, y_tol)


@pytest.mark.parametrize("t", [BF, F32])
@pytest.mark.parametrize("rows, width", [(1, 7), (300, 640), (9, 1337), (5, 4352)])
def test_outputs_that_are_not_wanted(dev, rows, width, t):
    """The C entry points without the mean, the deviation, or one of the parameters' gradients: the others are the same."""
    lib, none = B.library(), 0
    x, dy = randn(dev, 1, rows, width).to(t), randn(dev, 2, rows, width).to(t)
    w, b = 1 + 0.2 * randn(dev, 3, width), randn(dev, 4, width)
    want = mr.layer_norm_forward(x, w, b, 1e-5)
    stream = torch.cuda.current_stream().cuda_stream
    for with_mean, with_rstd in ((False, False), (True, False), (False, True)):
        y = torch.full_like(x, 7)
        mean, rstd = torch.full((rows,), 7.0, device=dev), torch.full((rows,), 7.0, device=dev)
        p = B.LayerNormProblem(rows, width, x.data_ptr(), width, none, 0, w.data_ptr(), b.data_ptr(), none, 0,
                               mean.data_ptr() if with_mean else none, rstd.data_ptr() if with_rstd else none,
                               y.data_ptr(), width, none, 0, none, 0, CODES[t], B.MR_F32, 0, 0, 1e-5)
        assert lib.layer_norm_forward(ctypes.addressof(p), stream) == 0
        assert torch.equal(y, want.y)
        assert torch.equal(mean, want.mean if with_mean else torch.full_like(mean, 7))
        assert torch.equal(rstd, want.rstd if with_rstd else torch.full_like(rstd, 7))
    both = mr.layer_norm_backward(dy, x, want.mean, want.rstd, w)
    _, _, dw, w_tol, db, b_tol = grad_reference(dy, x, want.mean, want.rstd, w, None)
    for with_dw, with_db in ((True, False), (False, True)):
        dx = torch.full_like(x, 7)
        dweight, dbias = torch.full((width,), 7.0, device=dev), torch.full((width,), 7.0, device=dev)
        p = B.LayerNormGradProblem(rows, width, dy.data_ptr(), width, x.data_ptr(), width, want.mean.data_ptr(),
                                   want.rstd.data_ptr(), w.data_ptr(), none, 0, dx.data_ptr(), width,
                                   dweight.data_ptr() if with_dw else none, dbias.data_ptr() if with_db else none, CODES[t],
                                   B.MR_F32)
        need = lib.layer_norm_backward_workspace(ctypes.addressof(p))
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
        assert lib.layer_norm_backward(ctypes.addressof(p), ws.data_ptr(), need, stream) == 0
        assert torch.equal(dx, both[0])
        for got, same, ref, tol, wanted in ((dweight, both[1], dw, w_tol, with_dw), (dbias, both[2], db, b_tol, with_db)):
            if wanted:
                assert torch.equal(got, same)
                within(got, ref, tol)
            else:
                assert bool((got == 7).all())
