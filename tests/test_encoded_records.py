"""Which record buffers an encoded matrix hands to the library (CPU: the
checks come before any device work)."""
import ctypes

import pytest
import torch

ROWS, COLS = 4, 64


@pytest.fixture(scope="module")
def e8q():
    from bit_e8_lattice_b200 import build, e8q

    build.build()
    return e8q


def matrix(e8q, esc, ovf, esc_count, ovf_count):
    ptr = torch.arange(ROWS + 1, dtype=torch.int64)
    m = e8q.Encoded(torch.zeros((ROWS, COLS // 8), dtype=torch.int16), torch.ones(ROWS), torch.ones(COLS, dtype=torch.int8),
                    esc, ptr, ovf, ptr, ROWS, COLS, 0, 0, esc_count, ovf_count)
    m.keep = ptr
    return m


def calls(e8q, m):
    """Every entry point that takes an encoded matrix, with buffers of its own."""
    L, c = e8q.lib(), ctypes.byref(m.c())
    vp, far = ctypes.c_void_p, [0x1000000000 * (i + 1) for i in range(4)]  # never dereferenced
    return dict(decode=L.e8q_decode(c, 2, vp(far[0]), None),
                decode_rows=L.e8q_decode_rows(c, 2, vp(far[1]), 1, 3, 0, 1.0, vp(far[0]), 1, None),
                gemv=L.e8q_dequant_gemv(c, vp(far[1]), 1, vp(far[0]), vp(far[2]), 1 << 40, None),
                gemm=L.e8q_dequant_gemm(c, vp(far[1]), 64, vp(far[0]), vp(far[2]), 1 << 40, None))


def some(size):
    return torch.zeros(8 * size, dtype=torch.uint8)


NONE = torch.zeros(0, dtype=torch.uint8)


@pytest.mark.parametrize("esc,ovf,counts", [(NONE, some(20), (4, 8)), (None, some(20), (4, 8)), (None, some(20), (0, 8)),
                                            (some(8), NONE, (8, 4)), (some(8), None, (8, 4)), (some(8), None, (8, 0)),
                                            (NONE, NONE, (4, 0)), (NONE, NONE, (0, 1)), (None, None, (0, 0))])
def test_row_pointers_without_their_records_are_refused(e8q, esc, ovf, counts):
    """Row pointers that claim records which nobody holds (a lost buffer): the
    weights would silently be other ones."""
    m = matrix(e8q, esc, ovf, *counts)
    c = m.c()
    for buffer, count, pointer in ((esc, counts[0], c.esc_row_ptr), (ovf, counts[1], c.ovf_row_ptr)):
        if buffer is None or buffer.numel() or count:
            assert pointer == m.keep.data_ptr()
    assert calls(e8q, m) == dict(decode=1, decode_rows=1, gemv=1, gemm=1)


def test_empty_record_buffers_that_claim_nothing(e8q):
    """A matrix whose records are none (gathered shards of one: empty buffers, counts 0)."""
    c = matrix(e8q, NONE, NONE, 0, 0).c()
    assert not c.esc and not c.ovf and not c.esc_row_ptr and not c.ovf_row_ptr
    c = matrix(e8q, some(8), some(20), 8, 8).c()
    assert c.esc and c.ovf and c.esc_row_ptr and c.ovf_row_ptr
