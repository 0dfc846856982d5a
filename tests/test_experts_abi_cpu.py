"""Refusals of the operators around a bank of experts, of layer norm and of
gradient clipping, none of which needs a GPU: the C entry points reject invalid
problems before anything is enqueued (they never dereference the device pointers
they are given), and the Python functions reject tensors that do not fit before
they call the library."""

import ctypes
import math

import pytest
import torch

from matrix_roots_amd import binding as B
from matrix_roots_amd import experts as X
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
    d = dict(rows=4, width=256, x=P[0], ldx=256, residual=P[1], ldres=256, weight=P[2], bias=P[9], h=P[3], ldh=256,
             mean=P[8], rstd=P[4], y=P[5], ldy=256, q=P[6], ldq=256, scales=P[7], lds=2, dtype=B.MR_BF16,
             w_dtype=B.MR_F32, q_dtype=B.MR_E4M3, eps=1e-6)
    d.update(kw)
    return B.LayerNormProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(rows=-1), SHAPE), (dict(rows=(1 << 30) + 1), SHAPE), (dict(width=0), SHAPE),
    (dict(width=16385, ldx=16385), SHAPE), (dict(dtype=B.MR_F64), PARAM), (dict(dtype=B.MR_E4M3), PARAM),
    (dict(w_dtype=B.MR_F16), PARAM), (dict(q_dtype=B.MR_BF16), PARAM), (dict(eps=-1.0), PARAM),
    (dict(eps=float("nan")), PARAM), (dict(eps=float("inf")), PARAM), (dict(y=0, q=0), NULL), (dict(weight=0), NULL),
    (dict(x=0), NULL), (dict(h=0), NULL), (dict(scales=0), NULL), (dict(ldx=255), STRIDE), (dict(ldh=255), STRIDE),
    (dict(lds=1), STRIDE), (dict(ldq=255), STRIDE), (dict(ldx=(1 << 22) + 8), STRIDE), (dict(x=P[0] + 1), PARAM),
    (dict(weight=P[2] + 2), PARAM), (dict(bias=P[9] + 2), PARAM), (dict(rstd=P[4] + 2), PARAM),
    (dict(mean=P[8] + 1), PARAM), (dict(scales=P[7] + 2), PARAM), (dict(h=P[0]), ALIAS), (dict(y=P[1] + 512), ALIAS),
    (dict(q=P[5]), ALIAS), (dict(mean=P[4] + 8), ALIAS), (dict(rstd=P[2]), ALIAS), (dict(y=P[9]), ALIAS),
    (dict(rows=0), OK),
])
def test_layer_norm_forward_refusals(lib, change, status):
    assert lib.layer_norm_forward(at(norm(**change)), None) == status
    assert status == OK or lib.mr_last_error_message()


def grad(**kw):
    d = dict(rows=4, width=256, dy=P[0], lddy=256, h=P[1], ldh=256, mean=P[7], rstd=P[2], weight=P[3], dresidual=P[4],
             ldres=256, dx=P[5], lddx=256, dweight=P[6], dbias=P[8], dtype=B.MR_F16, w_dtype=B.MR_F16)
    d.update(kw)
    return B.LayerNormGradProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(rows=-1), SHAPE), (dict(width=0), SHAPE), (dict(dtype=9), PARAM), (dict(w_dtype=B.MR_BF16), PARAM),
    (dict(dy=0), NULL), (dict(h=0), NULL), (dict(mean=0), NULL), (dict(rstd=0), NULL), (dict(weight=0), NULL),
    (dict(dx=0), NULL), (dict(lddy=128), STRIDE), (dict(ldres=128), STRIDE), (dict(dweight=P[6] + 1), PARAM),
    (dict(dbias=P[8] + 2), PARAM), (dict(dx=P[0]), ALIAS), (dict(dx=P[4]), ALIAS), (dict(dweight=P[5]), ALIAS),
    (dict(dbias=P[6] + 8), ALIAS), (dict(), WORKSPACE),
])
def test_layer_norm_backward_refusals(lib, change, status):
    p = grad(**change)
    ws = 0 if status == WORKSPACE else P[9]
    assert lib.layer_norm_backward(at(p), ws, 1 << 30, None) == status
    if status == WORKSPACE:
        need = lib.layer_norm_backward_workspace(at(p))
        assert need >= 2 * 256 * 4 and need % 256 == 0
        assert lib.layer_norm_backward(at(p), P[9], need - 1, None) == WORKSPACE
        assert lib.layer_norm_backward(at(p), P[9] + 8, need, None) == WORKSPACE
        assert lib.layer_norm_backward(at(p), P[5], need, None) == ALIAS
        assert lib.layer_norm_backward_workspace(at(grad(dweight=0))) == need
        assert lib.layer_norm_backward_workspace(at(grad(dweight=0, dbias=0))) == 0


def route(**kw):
    d = dict(tokens=8, experts=64, k=4, logits=P[0], ldl=64, chosen=P[1], weights=P[2], log_sum=P[3], dtype=B.MR_F32,
             normalize=1)
    d.update(kw)
    return B.RouteProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(tokens=-1), SHAPE), (dict(experts=0), SHAPE), (dict(experts=4097, ldl=4097), SHAPE), (dict(k=0), SHAPE),
    (dict(k=17), SHAPE), (dict(experts=3, k=4), SHAPE), (dict(tokens=1 << 30), SHAPE), (dict(dtype=B.MR_E4M3), PARAM),
    (dict(normalize=2), PARAM), (dict(logits=0), NULL), (dict(chosen=0), NULL), (dict(weights=0), NULL),
    (dict(log_sum=0), NULL), (dict(ldl=63), STRIDE), (dict(logits=P[0] + 2), PARAM), (dict(chosen=P[1] + 2), PARAM),
    (dict(chosen=P[0]), ALIAS), (dict(weights=P[1] + 64), ALIAS), (dict(log_sum=P[2]), ALIAS), (dict(tokens=0), OK),
])
def test_route_refusals(lib, change, status):
    assert lib.route_tokens(at(route(**change)), None) == status


def route_grad(**kw):
    d = dict(tokens=8, experts=64, k=4, logits=P[0], ldl=64, chosen=P[1], weights=P[2], dweights=P[4],
             dlogits=P[5], ldd=64, dtype=B.MR_BF16, normalize=0)
    d.update(kw)
    return B.RouteGradProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(tokens=-1), SHAPE), (dict(experts=0), SHAPE), (dict(k=17), SHAPE), (dict(dtype=B.MR_F64), PARAM),
    (dict(normalize=-1), PARAM), (dict(logits=0), NULL), (dict(chosen=0), NULL), (dict(weights=0), NULL),
    (dict(dweights=0), NULL), (dict(dlogits=0), NULL), (dict(ldd=63), STRIDE),
    (dict(dweights=P[4] + 1), PARAM), (dict(dlogits=P[0]), ALIAS), (dict(dlogits=P[4]), ALIAS), (dict(tokens=0), OK),
])
def test_route_grad_refusals(lib, change, status):
    assert lib.route_tokens_backward(at(route_grad(**change)), None) == status


def order(**kw):
    d = dict(tokens=8, experts=64, k=4, chosen=P[0], ldc=4, offsets=P[1], place=P[2], index_bits=32)
    d.update(kw)
    return B.OrderProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(tokens=-1), SHAPE), (dict(experts=0), SHAPE), (dict(experts=4097), SHAPE), (dict(k=0), SHAPE),
    (dict(k=65, ldc=65), SHAPE), (dict(tokens=1 << 29), SHAPE), (dict(index_bits=16), PARAM), (dict(chosen=0), NULL),
    (dict(offsets=0), NULL), (dict(place=0), NULL), (dict(ldc=3), STRIDE), (dict(index_bits=64, chosen=P[0] + 4), PARAM),
    (dict(place=P[0]), ALIAS), (dict(offsets=P[2] + 64), ALIAS), (dict(tokens=0, offsets=0), NULL),
])
def test_order_refusals(lib, change, status):
    assert lib.order_by_expert(at(order(**change)), P[9], 1 << 30, None) == status


def test_order_workspace(lib):
    assert lib.order_by_expert_workspace(at(order(tokens=4096, k=1, ldc=1))) == 0
    p = order(tokens=4097, k=1, ldc=1)
    need = lib.order_by_expert_workspace(at(p))
    assert need > 0 and need % 256 == 0
    assert lib.order_by_expert(at(p), None, 0, None) == WORKSPACE
    assert lib.order_by_expert(at(p), P[9], need - 1, None) == WORKSPACE
    assert lib.order_by_expert(at(p), P[2], need, None) == ALIAS
    # 256 workgroups' counts at most
    assert lib.order_by_expert_workspace(at(order(tokens=1 << 25, k=32, ldc=32))) <= 256 * 65 * 4 + 256


def dispatch(**kw):
    d = dict(tokens=8, experts=64, k=4, width=96, X=P[0], ldx=96, place=P[1], offsets=P[2], weights=P[3], Z=P[4], ldz=96,
             Y=P[5], ldy=96, dots=P[6], dtype=B.MR_BF16)
    d.update(kw)
    return B.DispatchProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(tokens=-1), SHAPE), (dict(experts=0), SHAPE), (dict(width=0), SHAPE), (dict(width=65537), SHAPE),
    (dict(k=65), SHAPE), (dict(dtype=B.MR_F64), PARAM), (dict(Z=0), NULL), (dict(dots=0), NULL),
    (dict(Z=0, dots=0), UNSUPPORTED), (dict(X=0), NULL), (dict(Y=0), NULL), (dict(place=0), NULL),
    (dict(offsets=0), NULL), (dict(ldx=95), STRIDE), (dict(ldy=95), STRIDE), (dict(ldz=95), STRIDE),
    (dict(weights=P[3] + 2), PARAM), (dict(Y=P[4]), ALIAS), (dict(Y=P[0] + 64), ALIAS), (dict(dots=P[3]), ALIAS),
    (dict(dots=P[5] + 32), ALIAS), (dict(tokens=0), OK),
])
def test_dispatch_refusals(lib, change, status):
    assert lib.dispatch_rows(at(dispatch(**change)), None) == status


def combine(**kw):
    d = dict(tokens=8, experts=64, k=4, width=96, Y=P[0], ldy=96, place=P[1], offsets=P[2], weights=P[3], residual=P[4],
             ldres=96, OUT=P[5], ldo=96, dtype=B.MR_F32)
    d.update(kw)
    return B.CombineProblem(**d)


@pytest.mark.parametrize("change, status", [
    (dict(tokens=-1), SHAPE), (dict(experts=4097), SHAPE), (dict(width=0), SHAPE), (dict(k=0), SHAPE),
    (dict(dtype=B.MR_E5M2), PARAM), (dict(Y=0), NULL), (dict(OUT=0), NULL), (dict(place=0), NULL),
    (dict(offsets=0), NULL), (dict(ldy=95), STRIDE), (dict(ldres=95), STRIDE), (dict(ldo=95), STRIDE),
    (dict(weights=P[3] + 1), PARAM), (dict(OUT=P[0]), ALIAS), (dict(OUT=P[4]), ALIAS), (dict(OUT=P[1]), ALIAS),
    (dict(tokens=0), OK),
])
def test_combine_refusals(lib, change, status):
    assert lib.combine_rows(at(combine(**change)), None) == status


def clip(**kw):
    d = dict(m=8, n=64, G=P[0], ldg=64, OUT=0, ldo=0, dtype=B.MR_BF16, out_dtype=B.MR_BF16)
    d.update(kw)
    return B.ClipProblem(**d)


def call_clip(lib, *probs, count=None, max_norm=1.0, norms=P[10], ws=P[9], ws_bytes=1 << 30):
    arr = (B.ClipProblem * max(len(probs), 1))(*probs)
    return lib.clip_gradients_batched(at(arr), len(probs) if count is None else count, max_norm, norms, ws, ws_bytes, None)


@pytest.mark.parametrize("change, status", [
    (dict(m=-1), SHAPE), (dict(n=-1), SHAPE), (dict(m=1 << 21, n=1 << 20), SHAPE), (dict(dtype=B.MR_F64), PARAM),
    (dict(G=0), NULL), (dict(ldg=63), STRIDE), (dict(ldg=1 << 40), STRIDE), (dict(G=P[0] + 1), PARAM),
    (dict(OUT=P[1], ldo=64, out_dtype=B.MR_F16), PARAM), (dict(OUT=P[1], ldo=63), STRIDE),
    (dict(OUT=P[1] + 2, ldo=64, out_dtype=B.MR_F32), PARAM), (dict(OUT=P[0], ldo=64), ALIAS), (dict(G=P[10]), ALIAS),
])
def test_clip_refusals(lib, change, status):
    assert call_clip(lib, clip(**change)) == status


def test_clip_refusals_of_a_call(lib):
    two = clip(), clip(G=P[0] + 16)
    assert call_clip(lib, *two) == ALIAS  # the same values twice
    assert call_clip(lib, clip(), count=-1) == PARAM
    assert call_clip(lib, clip(), max_norm=-1.0) == PARAM
    assert call_clip(lib, clip(), max_norm=math.nan) == PARAM
    assert call_clip(lib, clip(), norms=0) == NULL
    assert call_clip(lib, clip(), norms=P[10] + 4) == PARAM
    assert lib.clip_gradients_batched(None, 1, 1.0, P[10], P[9], 1 << 30, None) == NULL
    arr = (B.ClipProblem * 1)(clip())
    need = lib.clip_gradients_batched_workspace(at(arr), 1)
    assert need > 0 and need % 256 == 0
    assert call_clip(lib, clip(), ws=0, ws_bytes=0) == WORKSPACE
    assert call_clip(lib, clip(), ws_bytes=need - 1) == WORKSPACE
    assert call_clip(lib, clip(), ws=P[0]) == ALIAS
    assert call_clip(lib, clip(), ws=P[10]) == ALIAS
    assert lib.clip_gradients_batched_workspace(at(arr), 0) == 0
    # a few thousand partial sums for any amount of values
    big = (B.ClipProblem * 3)(*(clip(m=1 << 20, n=1 << 14, ldg=1 << 14) for _ in range(3)))
    assert lib.clip_gradients_batched_workspace(at(big), 3) < 1 << 16


def test_null_problems(lib):
    assert lib.layer_norm_forward(None, None) == NULL
    assert lib.layer_norm_backward(None, None, 0, None) == NULL
    assert lib.route_tokens(None, None) == NULL
    assert lib.route_tokens_backward(None, None) == NULL
    assert lib.order_by_expert(None, None, 0, None) == NULL
    assert lib.dispatch_rows(None, None) == NULL
    assert lib.combine_rows(None, None) == NULL


# ------------------------------------------------------- Python functions
def test_host_tensors_are_refused():
    x = torch.zeros(4, 8)
    i = torch.zeros(4, 2, dtype=torch.int32)
    o = X.ExpertOrder(torch.zeros(3, dtype=torch.int32), i)
    for call in (lambda: L.layer_norm_forward(x, torch.ones(8), None, 1e-6), lambda: X.route_tokens(x, 2),
                 lambda: X.order_by_expert(i, 2), lambda: X.dispatch_rows(x, o), lambda: X.combine_rows(x, o)):
        with pytest.raises(ValueError, match="GPU"):
            call()


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
    for module in (L, X):
        monkeypatch.setattr(module, "library", lambda: lib)
        monkeypatch.setattr(module, "_device", lambda *t: torch.device("cpu"))
        monkeypatch.setattr(module, "_stream", lambda stream, dev: 0)
        monkeypatch.setattr(module, "_in_use_on", lambda stream, *t: used.append((stream, [x for x in t if x is not None])))
    monkeypatch.setattr(B, "library", lambda: lib)
    monkeypatch.setattr(B, "_stream", lambda stream: 0)
    monkeypatch.setattr(B, "_current_gpu", lambda: -1)
    monkeypatch.setattr(B, "_in_use_on", lambda stream, *t: used.append((stream, [x for x in t if x is not None])))
    lib.used = used
    return lib


def test_what_does_not_fit_is_refused(fake):
    bf = torch.bfloat16
    x = torch.zeros(4, 8, dtype=bf)
    w = torch.ones(8)
    four = torch.ones(4)
    place = torch.zeros(4, 2, dtype=torch.int32)
    off = torch.zeros(3, dtype=torch.int32)
    o = X.ExpertOrder(off, place)
    y = torch.zeros(8, 8, dtype=bf)
    d = torch.zeros(4, 2)
    r = X.Routed(place, d, four)
    bad = [
        lambda: L.layer_norm_forward(x, torch.ones(7), None, 1e-6),
        lambda: L.layer_norm_forward(x, w, torch.ones(7), 1e-6),
        lambda: L.layer_norm_forward(x, w, w.bfloat16(), 1e-6),
        lambda: L.layer_norm_forward(x, w.half(), None, 1e-6),
        lambda: L.layer_norm_forward(x, w, w, 1e-6, residual=torch.zeros(4, 8)),
        lambda: L.layer_norm_forward(x, w, w, 1e-6, residual=torch.zeros(3, 8, dtype=bf)),
        lambda: L.layer_norm_forward(x, w, w, 1e-6, keep_y=False),
        lambda: L.layer_norm_forward(x, w, w, 1e-6, eight="e3m4"),
        lambda: L.layer_norm_forward(x.long(), w, w, 1e-6),
        lambda: L.layer_norm_forward(torch.zeros(8, 4, dtype=bf).t(), w, w, 1e-6),
        lambda: L.layer_norm_forward(x[0], w, w, 1e-6),
        lambda: L.layer_norm_backward(x, x.half(), four, four, w),
        lambda: L.layer_norm_backward(x, x, torch.ones(3), four, w),
        lambda: L.layer_norm_backward(x, x, four, four.double(), w),
        lambda: L.layer_norm_backward(x, x, four, four, w, dresidual=x[:2]),
        lambda: X.route_tokens(x.long(), 2),
        lambda: X.route_tokens(x[0], 2),
        lambda: X.route_tokens(torch.zeros(8, 4, dtype=bf).t(), 2),
        lambda: X.route_tokens_backward(d, x[:3], r),
        lambda: X.route_tokens_backward(d.half(), x, r),
        lambda: X.route_tokens_backward(d[:, :1], x, r),
        lambda: X.route_tokens_backward(d, x, X.Routed(place.long(), d, four)),
        lambda: X.route_tokens_backward(d.t().contiguous().t(), x, r),
        lambda: X.order_by_expert(x, 2),
        lambda: X.order_by_expert(place[0], 2),
        lambda: X.order_by_expert(place.t(), 2),
        lambda: X.dispatch_rows(x[:3], o),
        lambda: X.dispatch_rows(x.long(), o),
        lambda: X.dispatch_rows(x, X.ExpertOrder(off, place.long())),
        lambda: X.dispatch_rows(x, X.ExpertOrder(off.float(), place)),
        lambda: X.dispatch_rows(x, X.ExpertOrder(place, place)),
        lambda: X.combine_rows(y[:7], o),
        lambda: X.combine_rows(y[0], o),
        lambda: X.combine_rows(y, o, weights=d.double()),
        lambda: X.combine_rows(y, o, weights=d[:, :1]),
        lambda: X.combine_rows(y, o, residual=x.half()),
        lambda: X.combine_rows(y, o, residual=x[:, :7]),
        lambda: X.combine_rows_backward(x.half(), y, o, d),
        lambda: X.combine_rows_backward(x[:, :7], y, o, d),
        lambda: X.combine_rows_backward(x, y, o, d[:3]),
        lambda: B.clip_gradients_batched([], 1.0),
        lambda: B.clip_gradients_batched([x.long()], 1.0),
        lambda: B.clip_gradients_batched([x], 1.0, outs=[]),
        lambda: B.clip_gradients_batched([x], 1.0, outs=[torch.zeros(4, 7)]),
        lambda: B.clip_gradients_batched([x], 1.0, outs=[x.half()]),
        lambda: B.clip_gradients_batched([x], 1.0, outs=[torch.zeros(8, 4).t()]),
        lambda: B.clip_gradients_batched([torch.zeros(1, 8).expand(4, 8)], 1.0),
        lambda: B.clip_gradients_batched([torch.zeros(4, 8)[:, ::2]], 1.0),
        lambda: B.clip_gradients_batched([torch.zeros(4, 5, 8)[:, :3, :7]], 1.0),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            raise AssertionError(f"refusal {i} passed")
    assert fake.calls == []


def test_gradients_of_another_device_are_refused(fake, monkeypatch):
    monkeypatch.setattr(B, "_current_gpu", lambda: 0)
    with pytest.raises(ValueError, match="current GPU"):
        B.clip_gradients_batched([torch.zeros(4)], 1.0)
    assert fake.calls == []


def test_how_gradients_lie():
    big = torch.zeros(6, 10, 16)
    for t, want in [(big, (1, 960, 0)), (big[0], (1, 160, 0)), (big[0].t(), (1, 160, 0)), (big[:, :, :5], (60, 5, 16)),
                    (big[:, 0], (6, 16, 160)), (big[2:4], (1, 320, 0)), (big.permute(2, 0, 1), (1, 960, 0)),
                    (big[:, :3], (6, 48, 160)), (big[:1, :1, :1], (1, 1, 0)), (torch.zeros(()), (1, 1, 0)),
                    (torch.zeros(0, 4), (1, 0, 0)), (big[0, :, :5].t(), (10, 5, 16)), (big[:1, :, :5], (10, 5, 16))]:
        assert B._rows_of(t) == want, (t.shape, t.stride())


def test_buffers_are_marked_in_use_on_the_callers_stream(fake):
    s = Stream()
    bf = torch.bfloat16
    x, w, four = torch.zeros(4, 8, dtype=bf), torch.ones(8), torch.ones(4)
    r = L.layer_norm_forward(x, w, w, 1e-6, residual=x, eight="e4m3", stream=s)
    assert fake.used[-1][0] is s and len(fake.used[-1][1]) == 6 and r.h is not x
    L.layer_norm_backward(x, x, four, four, w, stream=s)
    assert len(fake.used[-1][1]) == 4  # workspace, dx, dweight, dbias
    r = X.route_tokens(x, 2, stream=s)
    assert len(fake.used[-1][1]) == 3
    X.route_tokens_backward(r.weights, x, r, stream=s)
    o = X.order_by_expert(r.experts, 8, stream=s)
    assert len(fake.used[-1][1]) == 3  # workspace, offsets, place
    y = X.dispatch_rows(x, o, stream=s)
    X.combine_rows(y, o, stream=s)
    X.combine_rows_backward(x, y, o, r.weights, stream=s)
    assert len(fake.used[-1][1]) == 2
    X.dispatch_rows_backward(y, o, stream=s)
    B.clip_gradients_batched([x, w], 1.0, stream=s)
    assert len(fake.used[-1][1]) == 2  # workspace, norms
    assert all(u[0] is s for u in fake.used)
    assert fake.calls == ["layer_norm_forward", "layer_norm_backward", "route_tokens", "route_tokens_backward",
                          "order_by_expert", "dispatch_rows", "combine_rows", "dispatch_rows", "combine_rows",
                          "clip_gradients_batched"]
