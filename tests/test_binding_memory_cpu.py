"""Where the binding takes new tensors from when it is called with `stream` (CPU
only: stand-ins for torch's streams and for the library).

A block of the current stream's pool may have been freed while work queued on
that stream still reads it; a kernel on another stream must not write there.  So
results and workspaces come from the memory of the stream that the kernels run
on, and results are marked as in use on the current stream, where they go."""

import contextlib

import pytest
import torch

from matrix_roots_amd import binding as B


class FakeStream:
    cuda_stream = 77


class FakeLib:
    """Accepts every call; workspace queries ask for 1 KiB."""

    def __getattr__(self, name):
        return (lambda *a: 1024) if name.endswith("_workspace") else (lambda *a: 0)


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

    def noting(make):
        def new(*a, **kw):
            t = make(*a, **kw)
            taken.append((t, now[-1]))
            return t

        return new

    monkeypatch.setattr(torch.cuda, "Stream", FakeStream)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[-1])
    monkeypatch.setattr(torch, "empty", noting(torch.empty))
    monkeypatch.setattr(torch, "empty_like", noting(torch.empty_like))
    monkeypatch.setattr(B, "_lib", FakeLib())
    monkeypatch.setattr(B, "_in_use_on", lambda s, *ts: marked.extend((t, s) for t in ts if t is not None and s is not None))
    return here, taken, marked


def calls():
    m, g, left, right = torch.eye(8), torch.zeros(8, 4), torch.eye(8), torch.eye(4)
    return {
        "quarter_root": lambda s: B.inv_quarter_root_batched([m, m], 1e-6, stream=s, return_info=False)[0],
        "sqrt_root": lambda s: B.inv_sqrt_root_batched([m], stream=s, return_info=False)[0],
        "polar": lambda s: B.polar_cans_batched([g, g], stream=s, return_info=False)[0],
        "hyperball": lambda s: [B.hyperball_update_batched([g], [g.clone()], 0.1, return_norms=True, stream=s)],
        "apply": lambda s: B.precondition_apply([left], [g], [right], stream=s),
    }


@pytest.mark.parametrize("name", list(calls()))
def test_new_tensors_come_from_the_calls_stream(streams, name):
    here, taken, marked = streams
    call = calls()[name]
    taken.clear()
    s = FakeStream()
    results = call(s)
    assert len(taken) > len(results)  # workspaces among them
    assert all(stream is s for _, stream in taken)
    for r in results:
        assert any(t is r and stream is here for t, stream in marked)


@pytest.mark.parametrize("name", list(calls()))
def test_without_a_stream_they_come_from_the_current_one(streams, name):
    here, taken, marked = streams
    call = calls()[name]
    taken.clear()
    call(None)
    assert taken and all(stream is here for _, stream in taken) and marked == []
