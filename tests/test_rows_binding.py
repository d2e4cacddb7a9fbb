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
