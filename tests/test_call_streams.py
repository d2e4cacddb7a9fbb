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


def adapters(e8q, tokens=200):
    a, b = torch.zeros((3, 8, 64), dtype=torch.bfloat16), torch.zeros((3, 40, 8), dtype=torch.bfloat16)
    op = e8q.Lora(a, b, torch.ones(3), tokens)
    op.device = torch.device("cuda", 0)
    return op


def run_adapters(op, tokens, stream):
    x, slots = torch.zeros((tokens, 64), dtype=torch.bfloat16), torch.zeros(tokens, dtype=torch.int32)
    y, u = op(x, slots, keep_u=True, stream=stream)
    return [y, u, *op.backward(y, x, u, slots, stream=stream)]


def run_rows(op, grad, ids, stream):
    return [op(grad, ids, stream=stream)]


@pytest.mark.parametrize("kind", ["adapters", "row gradient"])
def test_kept_memory_is_recorded_on_every_stream_that_uses_it(watched, kind):
    """The first call's stream owns it; a further one is recorded once, also when it is the current stream."""
    e8q, log = watched
    if kind == "adapters":
        op = adapters(e8q)

        def run(stream, tokens=200):
            return run_adapters(op, tokens, stream)
    else:
        op, grad, ids = rows_backward(e8q)

        def run(stream, tokens=200):
            return run_rows(op, grad[:tokens], ids[:tokens], stream)

    outs = run(SIDE)
    owned = [t for _, t in log.allocated]
    assert len(owned) == (7 if kind == "adapters" else 2) and all(s is SIDE for s, _ in log.allocated) and not log.recorded
    assert all(log.of(t) is SIDE for t in outs)

    def recorded():
        found = {(s.name, t.data_ptr()) for s, t in log.recorded}
        assert len(found) == len(log.recorded)
        log.recorded.clear()
        return found

    run(SIDE, 100)
    assert not recorded()
    run(None, 100)  # a smaller call on the current stream
    assert recorded() == {("main", t.data_ptr()) for t in owned}
    run(None)
    run(SIDE)
    assert not recorded()
    with torch.cuda.stream(THIRD):
        run(None)
    assert recorded() == {("third", t.data_ptr()) for t in owned}
    assert len(log.allocated) == len(owned)


class Library:
    """Answers every workspace question with 256 and every call with success, on the stream it is given."""

    def __init__(self, log):
        self.log = log

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return lambda *a: 256

        def call(*args):
            s = args[-1].value
            self.log.calls.append((name, next(x for x in (SIDE, self.log.main) if x.cuda_stream & (2 ** 64 - 1) == s)))
            return 0

        return call


@pytest.fixture
def library(watched, monkeypatch):
    e8q, log = watched
    log.main, log.written = log.current, []
    clone, copy, zeros = torch.Tensor.clone, torch.Tensor.copy_, torch.zeros
    note = log.written.append
    monkeypatch.setattr(e8q, "lib", lambda: Library(log))
    monkeypatch.setattr(torch.Tensor, "clone", lambda t: (note(log.current), clone(t))[1])
    monkeypatch.setattr(torch.Tensor, "copy_", lambda t, s: (note(log.current), copy(t, s))[1])
    monkeypatch.setattr(torch, "zeros", lambda *a, dtype=None, device=None: (note(log.current), zeros(*a, dtype=dtype))[1])
    return e8q, log


def encoded(e8q):
    some = torch.ones(8, dtype=torch.uint8)
    return e8q.Encoded(torch.ones((4, 8), dtype=torch.int16), torch.ones(4), torch.ones(64, dtype=torch.int8), some,
                       torch.ones(5, dtype=torch.int64), some, torch.ones(5, dtype=torch.int64), 4, 64, 0)


@pytest.mark.parametrize("stream", [SIDE, None])
@pytest.mark.parametrize("name", ["e8q_dequant_gemv", "e8q_dequant_gemm", "e8q_decode"])
def test_one_shot_calls_work_on_their_stream(library, name, stream):
    """Memory, kernels and the copy of the result on one stream."""
    e8q, log = library
    m, on = encoded(e8q), stream or log.main
    if name == "e8q_decode":
        e8q.e8q_decode(m, stream=stream)
    else:
        getattr(e8q, name)(m, torch.ones((2, 64), dtype=torch.bfloat16), stream=stream)
    assert log.calls == [(name, on)] and log.allocated and all(s is on for s, _ in log.allocated)
    assert all(s is on for s in log.written)


@pytest.mark.parametrize("stream", [SIDE, None])
def test_encode_with_given_scales_works_on_its_stream(library, stream):
    """The one-shot encode clears its outputs, and any encode copies the given
    scales, on the stream that the kernel runs on."""
    e8q, log = library
    w, signs, on = torch.ones((4, 64)), torch.ones(64, dtype=torch.int8), stream or log.main
    e8q.e8q_project_encode(w, signs, scales=[torch.ones(4)], esc_cap=64, ovf_cap=64, stream=stream)
    assert log.calls == [("e8q_project_encode", on)] and all(s is on for s, _ in log.allocated)
    assert len(log.written) == 3 and all(s is on for s in log.written)
    enc = e8q.Encoder([(4, 64)], [signs], torch.float32, scale_in=True, esc_cap=64, ovf_cap=64,
                      device="cpu")
    for run in (enc, enc.run_noalloc):
        log.written.clear()
        run([w], [torch.ones(4)], stream=stream)
        assert log.written == [on] and log.calls[-1][1] is on


@pytest.mark.parametrize("name", ["Gemv", "Gemm"])
def test_kept_memory_of_products_is_recorded(library, name):
    e8q, log = library
    op = getattr(e8q, name)(encoded(e8q), 2)
    x = torch.ones((2, 64), dtype=torch.bfloat16)
    op(x)
    assert not log.recorded
    y = op(x, stream=SIDE)
    op(x, stream=SIDE)
    assert len(log.allocated) == 2 and {t.data_ptr() for s, t in log.recorded if s is SIDE} == \
        {t.data_ptr() for _, t in log.allocated} == {y.data_ptr(), op.workspace.data_ptr()}
    assert len(log.recorded) == 2
    log.recorded.clear()
    op(x, out=torch.ones((2, 4), dtype=torch.bfloat16))
    assert not log.recorded
