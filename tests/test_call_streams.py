"""Which stream the memory that the binding allocates for a call belongs to
(CPU: a call on another stream would race with what the memory was freed
from, so the allocations are watched here, with no kernel).

torch's allocator hands a block out again in the order of the stream that it
was allocated on.  What a call on `stream` writes has to come from that
stream's memory, and memory of an object that is used on further streams has
to be recorded on them.
"""
import contextlib

import pytest
import torch


class Stream:
    def __init__(self, name):
        self.name = name
        self.cuda_stream = hash(name)

    def __repr__(self):
        return self.name


@pytest.fixture
def watched(monkeypatch):
    """The binding on CPU tensors without kernels; `log` has the stream of
    every allocation and the streams recorded on every tensor."""
    from bit_e8_lattice_b200 import build, e8q

    build.build()

    class Log:
        current = Stream("main")
        allocated = []   # (stream, tensor)
        recorded = []    # (stream, tensor)
        calls = []       # (entry point, stream)

        def of(self, t):
            """The stream that t's memory belongs to."""
            return next(s for s, a in self.allocated if a.untyped_storage().data_ptr() == t.untyped_storage().data_ptr())

    log = Log()
    log.allocated, log.recorded, log.calls = [], [], []
    empty = torch.empty

    @contextlib.contextmanager
    def on(stream):
        before, log.current = log.current, stream
        yield
        log.current = before

    def alloc(*size, dtype=None, device=None):
        t = empty(*size, dtype=dtype)
        log.allocated.append((log.current, t))
        return t

    def call(what, device, stream, *args):
        log.calls.append((what, stream if stream is not None else log.current))

    monkeypatch.setattr(torch, "empty", alloc)
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: log.current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: log.recorded.append((s, t)))
    monkeypatch.setattr(e8q, "_require", lambda *a: None)
    monkeypatch.setattr(e8q, "_require_cuda", lambda *a: None)
    monkeypatch.setattr(e8q, "_current_stream", lambda index: log.current.cuda_stream)
    monkeypatch.setattr(e8q, "_call", call)
    return e8q, log


SIDE, THIRD = Stream("side"), Stream("third")


def rows_backward(e8q, n=200):
    op = e8q.RowsBackward(10, 64, n, device=torch.device("cuda", 0))
    return op, torch.zeros((n, 64), dtype=torch.bfloat16), torch.zeros(n, dtype=torch.int64)


def test_row_gradient_memory_belongs_to_the_calls_stream(watched):
    e8q, log = watched
    op, grad, ids = rows_backward(e8q)
    out = op(grad, ids, stream=SIDE)
    assert log.calls == [("e8q_rows_backward", SIDE)] and len(log.allocated) == 2
    assert all(s is SIDE for s, _ in log.allocated) and log.of(out) is SIDE


def test_row_gradient_workspace_belongs_to_the_calls_stream(watched):
    e8q, log = watched
    op, grad, ids = rows_backward(e8q)
    op(grad, ids, torch.zeros((10, 64), dtype=torch.bfloat16), stream=SIDE)
    assert [s for s, _ in log.allocated] == [SIDE]
