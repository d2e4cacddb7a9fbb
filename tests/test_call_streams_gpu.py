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
