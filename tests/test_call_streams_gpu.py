"""Calls on a given stream whose memory the binding allocates: nothing that is
still queued on the current stream may write to it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def e8q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_e8_lattice_b200 import e8q as m

    m.init()
    return m


def freed_but_still_written(shape, dtype):
    """Memory that the current stream goes on writing after it was given back: the
    allocator may hand it to that stream at once, to others not."""
    t = torch.empty(shape, dtype=dtype, device="cuda")
    torch.cuda._sleep(100_000_000)  # some 50 ms
    t.fill_(float("nan"))
    del t


@pytest.mark.parametrize("n", [100, 300, 9000])
def test_row_gradient_on_another_stream(e8q, n):
    rows, cols = 600, 2048
    g = torch.Generator("cuda").manual_seed(n)
    grad = torch.randint(-4, 5, (n, cols), device="cuda", generator=g).bfloat16()
    ids = torch.randint(-1, rows, (n,), device="cuda", generator=g)
    want = e8q.e8q_rows_backward(grad, ids, rows)
    side = torch.cuda.Stream()
    op = e8q.RowsBackward(rows, cols, n)
    torch.cuda.synchronize()
    freed_but_still_written((rows, cols), torch.bfloat16)
    got = op(grad, ids, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("tokens", [90, 300])
def test_adapters_dropped_while_a_call_runs_on_another_stream(e8q, tokens):
    """The object's memory is the first call's stream's; the call that still
    runs is another stream's.  What is allocated meanwhile is other memory."""
    from test_lora_gpu import make

    d = make(tokens, 264, 136, 16, 5)
    op = e8q.Lora(d["a"], d["b"], d["scale"], tokens)
    y, u = (t.clone() for t in op(d["x"], d["slots"], base=d["base"], keep_u=True))
    grads = [t.clone() for t in op.backward(d["grad_y"], d["x"], u, d["slots"])]
    out, uo = torch.empty_like(y), torch.empty_like(u)
    got = [torch.empty_like(t) for t in grads]
    size = [t.numel() * t.element_size() for t, _ in op._kept._kept.values()]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    op(d["x"], d["slots"], base=d["base"], out=out, u=uo, stream=side)
    op.backward(d["grad_y"], d["x"], uo, d["slots"], grad_a=got[0], grad_b=got[1], grad_x=got[2], stream=side)
    del op
    fillers = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in size]
    torch.cuda.synchronize()
    assert torch.equal(out, y) and torch.equal(uo, u) and all(torch.equal(a, b) for a, b in zip(got, grads))
    assert all(bool((f == 255).all()) for f in fillers)


def test_row_gradient_dropped_while_a_call_runs_on_another_stream(e8q):
    n, rows, cols = 2000, 300, 1024
    grad, ids = torch.randn((n, cols), device="cuda").bfloat16(), torch.randint(0, rows, (n,), device="cuda")
    op = e8q.RowsBackward(rows, cols, n)
    want = op(grad, ids).clone()
    size = [t.numel() * t.element_size() for t, _ in op._kept._kept.values()]
    side = torch.cuda.Stream()
    got = torch.empty_like(want)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    op(grad, ids, got, stream=side)
    del op
    fillers = [torch.full((m,), 255, dtype=torch.uint8, device="cuda") for m in size]
    torch.cuda.synchronize()
    assert torch.equal(got, want) and all(bool((f == 255).all()) for f in fillers)
