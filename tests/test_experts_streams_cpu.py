"""Where layer norm, the operators around a bank of experts and gradient clipping
take new tensors from when they are called with `stream` (CPU only: stand-ins for
torch's streams and for the library): from the memory of the stream that the
kernels run on, results marked as in use on the current stream too."""

import contextlib

import pytest
import torch

from matrix_roots_amd import binding as B
from matrix_roots_amd import experts as X
from matrix_roots_amd import linear as L


class FakeStream:
    cuda_stream = 77


class FakeLib:
    """Returns MR_OK and 512-byte workspaces."""

    def __getattr__(self, name):
        return (lambda *a: 512) if name.endswith("_workspace") else (lambda *a: 0)


@pytest.fixture
def streams(monkeypatch):
    """(the current stream, [(tensor, the stream it was taken from)], [(storage, stream it is marked for)])"""
    here = FakeStream()
    now, taken, marked = [here], [], []

    @contextlib.contextmanager
    def on(stream):
        now.append(stream)
        yield
        now.pop()

    empty = torch.empty

    def new(*a, **kw):
        t = empty(*a, **kw)
        taken.append((t, now[-1]))
        return t

    def mark(stream, *tensors):
        if stream is not None:
            marked.extend((t.untyped_storage().data_ptr(), stream) for t in tensors if t is not None)

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch, "empty", new)
    for module in (B, L, X):
        monkeypatch.setattr(module, "library", lambda: FakeLib())
        monkeypatch.setattr(module, "_in_use_on", mark)
    monkeypatch.setattr(B, "_current_gpu", lambda: -1)
    for module in (L, X):
        monkeypatch.setattr(module, "_device", lambda *t: torch.device("cpu"))
        monkeypatch.setattr(module, "_stream", lambda stream, dev: 0)
    return here, taken, marked


def calls():
    bf = torch.bfloat16
    x, w, four = torch.zeros(4, 8, dtype=bf), torch.ones(8), torch.ones(4)
    chosen, d = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2)
    order, y = X.ExpertOrder(torch.zeros(9, dtype=torch.int32), chosen), torch.zeros(8, 8, dtype=bf)
    routed = X.Routed(chosen, d, four)
    return {
        "norm": lambda **k: L.layer_norm_forward(x, w, w, 1e-6, residual=x, eight="e4m3", **k),
        "norm_grad": lambda **k: L.layer_norm_backward(x, x, four, four, w, **k),
        "route": lambda **k: X.route_tokens(x, 2, **k),
        "route_grad": lambda **k: [X.route_tokens_backward(d, x, routed, **k)],
        "order": lambda **k: X.order_by_expert(chosen, 8, **k),
        "dispatch": lambda **k: [X.dispatch_rows(x, order, **k)],
        "dispatch_grad": lambda **k: [X.dispatch_rows_backward(y, order, **k)],
        "combine": lambda **k: [X.combine_rows(y, order, weights=d, residual=x, **k)],
        "combine_grad": lambda **k: X.combine_rows_backward(x, y, order, d, **k),
        "clip": lambda **k: B.clip_gradients_batched([x, y], 1.0, return_norms=True, **k),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_new_tensors_come_from_the_calls_stream(streams, name):
    here, taken, marked = streams
    call = calls()[name]
    taken.clear()
    s = FakeStream()
    results = call(stream=s)
    assert taken and all(stream is s for _, stream in taken)
    for r in results:
        assert (r.untyped_storage().data_ptr(), here) in marked


@pytest.mark.parametrize("name", [n for n in calls() if n != "clip"])
def test_without_a_stream_they_come_from_the_current_one(streams, name):
    here, taken, marked = streams
    call = calls()[name]
    taken.clear()
    call()
    assert taken and all(stream is here for _, stream in taken) and marked == []
