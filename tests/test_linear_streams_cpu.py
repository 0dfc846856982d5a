"""Where the linear-layer operators take new tensors from when they are called
with `stream` (CPU only: stand-ins for torch's streams and for the library).

A block of the current stream's pool may have been freed while work queued on
that stream still reads it; a kernel on another stream must not write there.  So
results and workspaces come from the memory of the stream that the kernels run
on, and results are marked as in use on the current stream, where they go."""

import contextlib

import pytest
import torch

from matrix_roots_amd import binding as B
from matrix_roots_amd import linear as L


class FakeStream:
    cuda_stream = 77


class FakeLib:
    """Returns MR_OK and 512-byte workspaces."""

    def __getattr__(self, name):
        return (lambda *a: 512) if name.endswith("_workspace") else (lambda *a: 0)


@pytest.fixture
def streams(monkeypatch):
    """(the current stream, [(tensor, the stream it was taken from)], [(tensor, stream it is marked for)])"""
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
            marked.extend((t, stream) for t in tensors if t is not None)

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch, "empty", new)
    for module in (B, L):
        monkeypatch.setattr(module, "library", lambda: FakeLib())
        monkeypatch.setattr(module, "_in_use_on", mark)
    monkeypatch.setattr(L, "_device", lambda *t: torch.device("cpu"))
    monkeypatch.setattr(L, "_stream", lambda stream, dev: 0)
    return here, taken, marked


def calls():
    bf = torch.bfloat16
    x, w, off = torch.zeros(4, 8, dtype=bf), torch.ones(8), torch.zeros(3, dtype=torch.int64)
    bank = torch.zeros(2, 16, 8, dtype=bf)
    a, s = torch.zeros(4, 8, dtype=torch.float8_e4m3fn), torch.ones(4, 1)
    return {
        "norm": lambda **k: L.rms_norm_forward(x, w, 1e-6, residual=x, eight="e4m3", **k),
        "norm_grad": lambda **k: L.rms_norm_backward(x, x, torch.ones(4), w, **k),
        "quantize": lambda **k: L.quantize_blocks(x, order="both", **k),
        "matmul": lambda **k: [L.block_scaled_matmul(a, s, a, s, **k)],
        "grouped": lambda **k: [L.grouped_matmul(x, bank, off, **k)],
        "grouped_grad": lambda **k: [L.grouped_weight_grad(x, x, off, **k)],
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
        assert any(t is r and stream is here for t, stream in marked)


@pytest.mark.parametrize("name", list(calls()))
def test_without_a_stream_they_come_from_the_current_one(streams, name):
    here, taken, marked = streams
    call = calls()[name]
    taken.clear()
    call()
    assert taken and all(stream is here for _, stream in taken) and marked == []


def test_a_callers_result_is_left_alone(streams):
    here, taken, marked = streams
    bf = torch.bfloat16
    x, out = torch.zeros(4, 8, dtype=bf), torch.zeros(4, 16, dtype=bf)
    taken.clear()
    L.grouped_matmul(x, torch.zeros(2, 16, 8, dtype=bf), torch.zeros(3, dtype=torch.int64), out=out, stream=FakeStream())
    assert taken == [] and marked == []
