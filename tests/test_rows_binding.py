"""What the binding of the row operators refuses before it calls the library (CPU)."""
import pytest
import torch


@pytest.fixture(scope="module")
def e8q():
    from bit_e8_lattice_b200 import build, e8q

    build.build()
    return e8q


def test_row_gradient_needs_a_cuda_device(e8q):
    """It took the GPU in place of another device."""
    with pytest.raises(e8q.E8qError, match="CUDA device"):
        e8q.RowsBackward(4, 8, 2, device="cpu")
    assert e8q.RowsBackward(4, 8, 2, device="cuda:0").device == torch.device("cuda", 0)


@pytest.mark.parametrize("first", [2 ** 63, -2 ** 63 - 1, 2 ** 64, 2 ** 64 + 3])
def test_first_row_outside_64_bits(e8q, first, monkeypatch):
    """ctypes drops the upper bits of a whole number: the rows would be other ones."""
    monkeypatch.setattr(e8q, "_require", lambda *a: None)
    monkeypatch.setattr(e8q, "_call", lambda *a: pytest.fail("called"))
    monkeypatch.setattr(e8q, "_current_stream", lambda index: 0)
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, dtype=None, device=None: empty(*a, dtype=dtype))
    some = torch.ones(8, dtype=torch.uint8)
    m = e8q.Encoded(torch.ones((4, 1), dtype=torch.int16), torch.ones(4), torch.ones(8, dtype=torch.int8), some,
                    torch.zeros(5, dtype=torch.int64), some, torch.zeros(5, dtype=torch.int64), 4, 8, 0)
    ids, grad = torch.zeros(2, dtype=torch.int64), torch.zeros((2, 8), dtype=torch.bfloat16)
    with pytest.raises(e8q.E8qError, match="first_row"):
        e8q.e8q_decode_rows(m, ids, first_row=first)
    with pytest.raises(e8q.E8qError, match="first_row"):
        e8q.RowsBackward(4, 8, 2, device="cuda:0")(grad, ids, first_row=first)
