"""Refusals of the linear-layer operators, none of which needs a GPU: the C
entry points reject invalid problems before anything is enqueued (they never
dereference the device pointers they are given), and the Python functions
reject tensors that do not fit before they call the library."""

import ctypes

import pytest
import torch

from matrix_roots_amd import binding as B
from matrix_roots_amd import linear as L

# fake, never-dereferenced "device" addresses, far apart and 256-byte aligned
P = [0x100000000 * k for k in range(1, 12)]
OK, NULL, SHAPE, STRIDE, PARAM, WORKSPACE, UNSUPPORTED, ALIAS = 0, 1, 2, 3, 4, 5, 7, 8


@pytest.fixture(scope="module")
def lib():
    return B.library()


def at(p):
    return ctypes.addressof(p)


def norm(**kw):
    d = dict(rows=4, width=256, x=P[0], ldx=256, residual=P[1], ldres=256, weight=P[2], h=P[3], ldh=256, rstd=P[4],
             y=P[5], ldy=256, q=P[6], ldq=256, scales=P[7], lds=2, dtype=B.MR_BF16, w_dtype=B.MR_F32,
             q_dtype=B.MR_E4M3, eps=1e-6)
    d.update(kw)
    return B.RmsNormProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(rows=-1), SHAPE), (dict(width=0), SHAPE), (dict(width=16385, ldx=16385), SHAPE),
    (dict(dtype=B.MR_F64), PARAM), (dict(dtype=B.MR_E4M3), PARAM), (dict(w_dtype=B.MR_F16), PARAM),
    (dict(q_dtype=B.MR_BF16), PARAM), (dict(eps=-1.0), PARAM), (dict(eps=float("nan")), PARAM),
    (dict(eps=float("inf")), PARAM), (dict(y=0, q=0), NULL), (dict(weight=0), NULL), (dict(x=0), NULL),
    (dict(h=0), NULL), (dict(scales=0), NULL), (dict(ldx=255), STRIDE), (dict(ldh=255), STRIDE),
    (dict(lds=1), STRIDE), (dict(ldq=255), STRIDE), (dict(ldx=(1 << 22) + 8), STRIDE), (dict(x=P[0] + 1), PARAM),
    (dict(weight=P[2] + 2), PARAM), (dict(rstd=P[4] + 2), PARAM), (dict(scales=P[7] + 2), PARAM),
    (dict(h=P[0]), ALIAS), (dict(y=P[1] + 512), ALIAS), (dict(q=P[5]), ALIAS), (dict(scales=P[6] + 128), ALIAS),
    (dict(rstd=P[2]), ALIAS), (dict(rows=0), OK),
])
def test_norm_forward_refusals(lib, change, status):
    assert lib.rms_norm_forward(at(norm(**change)), None) == status
    assert status == OK or lib.mr_last_error_message()


def grad(**kw):
    d = dict(rows=4, width=256, dy=P[0], lddy=256, h=P[1], ldh=256, rstd=P[2], weight=P[3], dresidual=P[4], ldres=256,
             dx=P[5], lddx=256, dweight=P[6], dtype=B.MR_F16, w_dtype=B.MR_F16)
    d.update(kw)
    return B.RmsNormGradProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(rows=-1), SHAPE), (dict(width=0), SHAPE), (dict(dtype=9), PARAM), (dict(w_dtype=B.MR_BF16), PARAM),
    (dict(dy=0), NULL), (dict(h=0), NULL), (dict(rstd=0), NULL), (dict(weight=0), NULL), (dict(dx=0), NULL),
    (dict(lddy=128), STRIDE), (dict(ldres=128), STRIDE), (dict(dweight=P[6] + 1), PARAM), (dict(dx=P[0]), ALIAS),
    (dict(dx=P[4]), ALIAS), (dict(dweight=P[5]), ALIAS), (dict(), WORKSPACE),
])
def test_norm_backward_refusals(lib, change, status):
    p = grad(**change)
    ws = 0 if status == WORKSPACE else P[9]
    assert lib.rms_norm_backward(at(p), ws, 1 << 30, None) == status
    if status == WORKSPACE:
        need = lib.rms_norm_backward_workspace(at(p))
        assert need >= 256 * 4 and need % 256 == 0
        assert lib.rms_norm_backward(at(p), P[9], need - 1, None) == WORKSPACE
        assert lib.rms_norm_backward(at(p), P[9] + 8, need, None) == WORKSPACE
        assert lib.rms_norm_backward(at(p), P[5], need, None) == ALIAS
        assert lib.rms_norm_backward_workspace(at(grad(dweight=0))) == 0


def quant(**kw):
    d = dict(m=256, n=384, X=P[0], ldx=384, Q=P[1], ldq=384, S=P[2], lds=3, QT=P[3], ldqt=256, ST=P[4], ldst=2,
             x_dtype=B.MR_F32, q_dtype=B.MR_E5M2, block=B.MR_BLOCK_SQUARE)
    d.update(kw)
    return B.QuantizeProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(m=-1), SHAPE), (dict(n=0), SHAPE), (dict(n=65537, ldx=65537), SHAPE), (dict(x_dtype=B.MR_E4M3), PARAM),
    (dict(q_dtype=B.MR_F16), PARAM), (dict(block=2), PARAM), (dict(Q=0, QT=0), NULL), (dict(X=0), NULL),
    (dict(S=0), NULL), (dict(ST=0), NULL), (dict(ldqt=255), STRIDE), (dict(ldst=1), STRIDE), (dict(X=P[0] + 2), PARAM),
    (dict(S=P[2] + 1), PARAM), (dict(Q=P[0]), ALIAS), (dict(QT=P[1] + 1), ALIAS), (dict(ST=P[2]), ALIAS),
    (dict(m=0), OK),
])
def test_quantize_refusals(lib, change, status):
    assert lib.quantize_blocks(at(quant(**change)), None) == status


def product(**kw):
    d = dict(m=256, n=128, k=256, A=P[0], lda=256, SA=P[1], ldsa=2, B=P[2], ldb=256, SB=P[3], ldsb=2, C=P[4], ldc=128,
             a_dtype=B.MR_E5M2, b_dtype=B.MR_E4M3, c_dtype=B.MR_F32, a_block=0, b_block=1, accumulate=0)
    d.update(kw)
    return B.ScaledMatmulProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(m=-1), SHAPE), (dict(n=0), SHAPE), (dict(k=0), SHAPE), (dict(k=(1 << 22) + 1), SHAPE),
    (dict(a_dtype=B.MR_F16), PARAM), (dict(b_dtype=B.MR_E5M2), UNSUPPORTED), (dict(b_dtype=0), PARAM),
    (dict(c_dtype=B.MR_E4M3), PARAM), (dict(a_block=2), PARAM), (dict(b_block=-1), PARAM), (dict(A=0), NULL),
    (dict(B=0), NULL), (dict(SA=0), NULL), (dict(SB=0), NULL), (dict(C=0), NULL), (dict(lda=255), STRIDE),
    (dict(ldsa=1), STRIDE), (dict(ldc=127), STRIDE), (dict(C=P[4] + 2), PARAM), (dict(SA=P[1] + 2), PARAM),
    (dict(C=P[0]), ALIAS), (dict(C=P[3]), ALIAS), (dict(m=0), OK),
])
def test_product_refusals(lib, change, status):
    assert lib.block_scaled_matmul(at(product(**change)), None, 0, None) == status


def test_product_workspace_is_asked_for(lib):
    p = product(m=128, n=128, k=16384, lda=16384, ldb=16384, ldsa=128, ldsb=128)
    need = lib.block_scaled_matmul_workspace(at(p))
    assert need > 0 and need % 256 == 0  # one tile of C, a long contraction: split
    assert lib.block_scaled_matmul(at(p), None, 0, None) == WORKSPACE
    assert lib.block_scaled_matmul(at(p), P[8], need - 1, None) == WORKSPACE
    assert lib.block_scaled_matmul(at(p), P[4], need, None) == ALIAS
    assert lib.block_scaled_matmul_workspace(at(product(m=8192, n=8192, ldc=8192))) == 0


def group(**kw):
    d = dict(experts=4, rows=64, n=96, k=160, X=P[0], ldx=160, W=P[1], ldw=160, w_stride=96 * 160, offsets=P[2], Y=P[3],
             ldy=96, dtype=B.MR_BF16, y_dtype=B.MR_F32, offset_bits=32, transpose=0)
    d.update(kw)
    return B.GroupedProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(experts=0), SHAPE), (dict(experts=4097), SHAPE), (dict(rows=-1), SHAPE), (dict(n=0), SHAPE),
    (dict(k=65537), SHAPE), (dict(dtype=B.MR_F32), PARAM), (dict(y_dtype=B.MR_F16), PARAM), (dict(offset_bits=16), PARAM),
    (dict(transpose=2), PARAM), (dict(offsets=0), NULL), (dict(X=0), NULL), (dict(W=0), NULL), (dict(Y=0), NULL),
    (dict(ldx=159), STRIDE), (dict(ldw=159), STRIDE), (dict(w_stride=96 * 160 - 1), STRIDE), (dict(ldy=95), STRIDE),
    (dict(offsets=P[2] + 2), PARAM), (dict(offset_bits=64, offsets=P[2] + 4), PARAM), (dict(Y=P[0]), ALIAS),
    (dict(Y=P[1] + 8), ALIAS), (dict(Y=P[2]), ALIAS), (dict(transpose=1), STRIDE), (dict(rows=0), OK),
])
def test_grouped_refusals(lib, change, status):
    assert lib.grouped_matmul(at(group(**change)), None) == status


def group_grad(**kw):
    d = dict(experts=4, rows=64, n=96, k=160, DY=P[0], lddy=96, X=P[1], ldx=160, offsets=P[2], DW=P[3], lddw=160,
             dw_stride=96 * 160, dtype=B.MR_F16, dw_dtype=B.MR_F32, offset_bits=64, accumulate=0)
    d.update(kw)
    return B.GroupedGradProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(experts=0), SHAPE), (dict(rows=-1), SHAPE), (dict(dtype=B.MR_F32), PARAM), (dict(dw_dtype=B.MR_BF16), PARAM),
    (dict(offset_bits=0), PARAM), (dict(DY=0), NULL), (dict(X=0), NULL), (dict(DW=0), NULL), (dict(offsets=0), NULL),
    (dict(lddy=95), STRIDE), (dict(lddw=159), STRIDE), (dict(dw_stride=1), STRIDE), (dict(DW=P[0]), ALIAS),
    (dict(DW=P[2]), ALIAS), (dict(DW=P[3] + 2), PARAM),
])
def test_grouped_grad_refusals(lib, change, status):
    assert lib.grouped_weight_grad(at(group_grad(**change)), None) == status


def test_null_problems(lib):
    assert lib.rms_norm_forward(None, None) == NULL
    assert lib.rms_norm_backward(None, None, 0, None) == NULL
    assert lib.quantize_blocks(None, None) == NULL
    assert lib.block_scaled_matmul(None, None, 0, None) == NULL
    assert lib.grouped_matmul(None, None) == NULL
    assert lib.grouped_weight_grad(None, None) == NULL


# ------------------------------------------------------- Python functions
def test_host_tensors_are_refused():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="GPU"):
        L.rms_norm_forward(x, torch.ones(8), 1e-6)
    with pytest.raises(ValueError, match="GPU"):
        L.quantize_blocks(x)


class Recorder:
    """Stands in for the library: records calls, returns MR_OK and 512-byte workspaces."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*a):
            if name.endswith("_workspace"):
                return 512
            self.calls.append(name)
            return 0

        return call


class Stream:
    cuda_stream = 77


@pytest.fixture
def fake(monkeypatch):
    lib = Recorder()
    used = []
    monkeypatch.setattr(L, "library", lambda: lib)
    monkeypatch.setattr(L, "_device", lambda *t: torch.device("cpu"))
    monkeypatch.setattr(L, "_stream", lambda stream, dev: 0)
    monkeypatch.setattr(L, "_in_use_on", lambda stream, *t: used.append((stream, [x for x in t if x is not None])))
    lib.used = used
    return lib


def test_what_does_not_fit_is_refused(fake):
    f32, bf = torch.float32, torch.bfloat16
    x = torch.zeros(4, 8, dtype=bf)
    w = torch.ones(8)
    off = torch.zeros(3, dtype=torch.int32)
    bank = torch.zeros(2, 16, 8, dtype=bf)
    e4, e5 = torch.float8_e4m3fn, torch.float8_e5m2
    a, b, s = torch.zeros(4, 8, dtype=e4), torch.zeros(6, 8, dtype=e4), torch.ones(4, 1)
    bad = [
        lambda: L.rms_norm_forward(x, torch.ones(7), 1e-6),
        lambda: L.rms_norm_forward(x, w.half(), 1e-6),
        lambda: L.rms_norm_forward(x, w, 1e-6, residual=torch.zeros(4, 8)),
        lambda: L.rms_norm_forward(x, w, 1e-6, residual=torch.zeros(3, 8, dtype=bf)),
        lambda: L.rms_norm_forward(x, w, 1e-6, keep_y=False),
        lambda: L.rms_norm_forward(x, w, 1e-6, eight="e3m4"),
        lambda: L.rms_norm_forward(x.long(), w, 1e-6),
        lambda: L.rms_norm_forward(torch.zeros(8, 4, dtype=bf).t(), w, 1e-6),
        lambda: L.rms_norm_backward(x, x.half(), torch.ones(4), w),
        lambda: L.rms_norm_backward(x, x, torch.ones(3), w),
        lambda: L.rms_norm_backward(x, x, torch.ones(4), w, dresidual=x[:2]),
        lambda: L.quantize_blocks(x, "e4m3", block="row"),
        lambda: L.quantize_blocks(x, "e4m3", order="all"),
        lambda: L.quantize_blocks(x, "int8"),
        lambda: L.block_scaled_matmul(a, s, b[:, :7], torch.ones(6, 1)),
        lambda: L.block_scaled_matmul(a, s, b, torch.ones(5, 1)),
        lambda: L.block_scaled_matmul(a, s.half(), b, torch.ones(6, 1)),
        lambda: L.block_scaled_matmul(x, s, b, torch.ones(6, 1)),
        lambda: L.block_scaled_matmul(a, s, b, torch.ones(6, 1), accumulate=True),
        lambda: L.block_scaled_matmul(a, s, b, torch.ones(6, 1), out=torch.zeros(4, 5)),
        lambda: L.grouped_matmul(x, bank.half(), off),
        lambda: L.grouped_matmul(x, bank, off[:2]),
        lambda: L.grouped_matmul(x, bank, off.float()),
        lambda: L.grouped_matmul(x, bank, off, transpose=True),
        lambda: L.grouped_matmul(x, bank.transpose(1, 2), off),
        lambda: L.grouped_matmul(x, bank[0], off),
        lambda: L.grouped_weight_grad(x, x[:3], off),
        lambda: L.grouped_weight_grad(x, x.half(), off),
        lambda: L.grouped_weight_grad(x, x, off, accumulate=True),
        lambda: L.grouped_weight_grad(x, x, off, out=torch.zeros(2, 8, 7)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises((ValueError, IndexError)):
            call()
            raise AssertionError(f"refusal {i} passed")
    assert fake.calls == []
    assert e5 not in (a.dtype, f32)


def test_buffers_are_marked_in_use_on_the_callers_stream(fake):
    s = Stream()
    bf = torch.bfloat16
    x = torch.zeros(4, 8, dtype=bf)
    r = L.rms_norm_forward(x, torch.ones(8), 1e-6, residual=x, eight="e4m3", stream=s)
    assert fake.used[-1][0] is s and len(fake.used[-1][1]) == 5 and r.h is not x
    L.rms_norm_backward(x, x, torch.ones(4), torch.ones(8), stream=s)
    assert len(fake.used[-1][1]) == 3  # workspace, dx, dweight
    q = L.quantize_blocks(x, order="both", stream=s)
    assert len(fake.used[-1][1]) == 4 and q.qt.stride(0) == 16
    L.block_scaled_matmul(q.q, q.scales, q.q, q.scales, stream=s)
    assert len(fake.used[-1][1]) == 2  # workspace and the result
    off = torch.zeros(3, dtype=torch.int64)
    L.grouped_matmul(x, torch.zeros(2, 16, 8, dtype=bf), off, stream=s)
    L.grouped_weight_grad(x, x, off, stream=s)
    assert all(u[0] is s for u in fake.used)
    assert fake.calls == ["rms_norm_forward", "rms_norm_backward", "quantize_blocks", "block_scaled_matmul",
                          "grouped_matmul", "grouped_weight_grad"]


def test_operands_of_other_dimensions_are_refused(fake):
    x, w, off = torch.zeros(4, 8).bfloat16(), torch.zeros(2, 8, 8).bfloat16(), torch.zeros(3, dtype=torch.int32)
    for call in (lambda: L.grouped_weight_grad(x[0], x, off), lambda: L.grouped_weight_grad(x, x[0], off),
                 lambda: L.grouped_weight_grad(x, x, off[0]), lambda: L.grouped_matmul(x, w, off[0]),
                 lambda: L.grouped_matmul(x[0, 0], w, off), lambda: L.grouped_matmul(x, w[0], off),
                 lambda: L.quantize_blocks(x[0]), lambda: L.rms_norm_forward(x[0], x[0], 1e-6),
                 lambda: L.rms_norm_backward(x[0], x[0], x[0].float(), x[0])):
        with pytest.raises(ValueError):
            call()
