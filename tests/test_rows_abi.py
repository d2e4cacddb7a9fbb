"""Argument checks of the row operators, before any device work (CPU)."""
import ctypes

import pytest

vp, P = ctypes.c_void_p, 0x100000


@pytest.fixture(scope="module")
def lib():
    from bit_e8_lattice_b200 import build, e8q

    build.build()
    return e8q.lib()


def matrix(rows=4, cols=64, block=0, **kw):
    from bit_e8_lattice_b200 import e8q

    m = e8q.EncodedC(P, P, P, None, None, None, None, 0, 0, rows, cols, 0, block, 0)
    for k, v in kw.items():
        setattr(m, k, v)
    return m


@pytest.mark.parametrize("change,expect", [
    (dict(basis=0), 1), (dict(basis=3), 1), (dict(ids=None), 1), (dict(ids=P + 4), 1), (dict(ids=P + 2, id_type=0), 1),
    (dict(id_type=2), 1), (dict(id_type=-1), 1), (dict(n=-1), 1), (dict(n=(1 << 30) + 1), 2),
    (dict(alpha=float("nan")), 1), (dict(alpha=float("inf")), 1), (dict(out=None), 1), (dict(out=P + 8), 1),
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(m=dict(cols=12)), 1), (dict(m=dict(cols=16392)), 2),
    (dict(m=dict(cols=64, block=128)), 1), (dict(m=dict(rows=-1)), 1), (dict(m=dict(signs=None)), 1),
    (dict(m=dict(signs=P + 4)), 1), (dict(m=dict(idx=None)), 1), (dict(m=dict(idx=P + 1)), 1),
    (dict(m=dict(scale=P + 2)), 1), (dict(m=dict(esc_row_ptr=P)), 1), (dict(m=dict(esc_row_ptr=P, esc=P + 4)), 1),
    (dict(m=dict(ovf_row_ptr=P, ovf=P + 2)), 1), (dict(m=dict(group_base=-1)), 1), (dict(n=0), 0),
    (dict(n=0, ids=None, out=None), 0), (dict(out=P + 16), 1),  # the ids inside out
])
def test_decode_rows_refusals(lib, change, expect):
    a = dict(m={}, basis=2, ids=P, id_type=1, n=3, first=0, alpha=1.0, out=0x200000, dtype=1)
    a.update(change)
    rc = lib.e8q_decode_rows(ctypes.byref(matrix(**a["m"])), a["basis"], vp(a["ids"]), a["id_type"], a["n"], a["first"],
                             a["alpha"], vp(a["out"]), a["dtype"], None)
    assert rc == expect
    assert lib.e8q_decode_rows(None, 2, vp(P), 1, 3, 0, 1.0, vp(P), 1, None) == 1


@pytest.mark.parametrize("change,expect", [
    (dict(grad=None), 1), (dict(grad=P + 8), 1), (dict(gd=2), 1), (dict(ld=-1), 1), (dict(ids=None), 1),
    (dict(ids=P + 4), 1), (dict(id_type=7), 1), (dict(n=-1), 1), (dict(n=(1 << 30) + 1), 2), (dict(rows=-1), 1),
    (dict(rows=(1 << 30) + 1), 2), (dict(cols=12), 1), (dict(cols=0), 1), (dict(cols=16392), 2),
    (dict(alpha=float("nan")), 1), (dict(acc=2), 1), (dict(acc=-1), 1), (dict(latent=None), 1),
    (dict(latent=P + 2), 1), (dict(latent=P + 16), 1),  # overlaps grad_out
    (dict(ids=0x40000000 + 64), 1),                     # ids inside the latents' gradient
    (dict(n=200, ws=None), 4), (dict(n=200, ws_bytes=64), 4), (dict(n=200, ws=P + 128), 4),
    (dict(rows=0), 0), (dict(n=0, acc=1), 0),
])
def test_rows_backward_refusals(lib, change, expect):
    a = dict(grad=P, gd=1, ids=0x200000, id_type=1, n=3, first=0, alpha=1.0, acc=0, latent=0x40000000, ld=1, rows=100,
             cols=64, ws=0x300000, ws_bytes=1 << 40)
    a.update(change)
    rc = lib.e8q_rows_backward(vp(a["grad"]), a["gd"], vp(a["ids"]), a["id_type"], a["n"], a["first"], a["alpha"],
                               a["acc"], vp(a["latent"]), a["ld"], a["rows"], a["cols"], vp(a["ws"]), a["ws_bytes"], None)
    assert rc == expect


def test_rows_backward_workspace_grows_with_the_ids(lib):
    """A workspace for n ids serves any smaller number of them."""
    f = lib.e8q_rows_backward_workspace_bytes
    for cols in (8, 1000, 1024, 2048, 14336, 16384):
        sizes = list(range(0, 12000, 37)) + [128, 129, 8192, 8193, 65536, 1 << 20]
        got = [f(n, cols) for n in sorted(sizes)]
        assert got == sorted(got) and all(b % 256 == 0 for b in got)
        assert f(200, cols) >= 8 * 200 and f(1 << 20, cols) >= 16 << 20
    for n, cols in ((-1, 64), (5, 12), (5, 16392), ((1 << 30) + 1, 64)):
        assert f(n, cols) == 256
