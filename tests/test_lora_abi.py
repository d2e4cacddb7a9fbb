"""Argument checks of the adapters, before any device work (CPU)."""
import ctypes

import pytest

vp, P = ctypes.c_void_p, 0x100000
FAR = [0x1000000000 * (i + 1) for i in range(12)]  # addresses far apart, never dereferenced


@pytest.fixture(scope="module")
def lib():
    from bit_e8_lattice_b200 import build, e8q

    build.build()
    return e8q.lib()


def adapters(**kw):
    from bit_e8_lattice_b200 import e8q

    a = e8q.AdaptersC(FAR[0], FAR[1], FAR[2], 128, 64, 4, 16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


BAD = [(dict(rows=12), 1), (dict(cols=4), 1), (dict(rank=4), 1), (dict(rank=12), 1), (dict(rows=0), 1), (dict(cols=-8), 1),
       (dict(rank=0), 1), (dict(n=-1), 1), (dict(n=2049), 2), (dict(rank=136), 2), (dict(rows=(1 << 20) + 8), 2),
       (dict(cols=(1 << 20) + 8), 2), (dict(a=None), 1), (dict(b=None), 1), (dict(scale=None), 1), (dict(a=FAR[0] + 8), 1),
       (dict(b=FAR[1] + 2), 1), (dict(scale=FAR[2] + 2), 1)]


def test_struct_size_matches_header():
    from bit_e8_lattice_b200 import e8q

    assert ctypes.sizeof(e8q.AdaptersC) == 48


@pytest.mark.parametrize("ad,expect", BAD)
def test_adapters_refusals(lib, ad, expect):
    a = ctypes.byref(adapters(**ad))
    assert lib.e8q_lora(a, vp(FAR[3]), vp(FAR[4]), 5, None, vp(FAR[5]), None, vp(P), 1 << 40, None) == expect
    assert lib.e8q_lora_backward(a, vp(FAR[3]), vp(FAR[4]), vp(FAR[5]), vp(FAR[6]), 5, vp(FAR[7]), vp(FAR[8]), None, None,
                                 vp(P), 1 << 40, None) == expect
    if expect == 2 or not {"a", "b", "scale"} & set(ad):
        assert lib.e8q_lora_workspace_bytes(a, 5, 0) == 256


@pytest.mark.parametrize("change,expect", [
    (dict(x=None), 1), (dict(x=FAR[3] + 8), 1), (dict(slots=None), 1), (dict(slots=FAR[4] + 2), 1), (dict(y=None), 1),
    (dict(y=FAR[5] + 2), 1), (dict(base=FAR[6] + 4), 1), (dict(u=FAR[7] + 4), 1), (dict(tokens=-1), 1),
    (dict(tokens=65537), 2), (dict(base=FAR[5] + 16), 1), (dict(y=FAR[3] + 16), 1), (dict(u=FAR[5]), 1), (dict(u=FAR[3]), 1),
    (dict(y=FAR[4]), 1), (dict(ws=None), 4), (dict(ws=P + 128), 4), (dict(ws_bytes=255), 4), (dict(tokens=0), 0),
    (dict(tokens=0, x=None, y=None, slots=None, ws=None), 0),
])
def test_lora_refusals(lib, change, expect):
    a = dict(x=FAR[3], slots=FAR[4], tokens=5, base=FAR[6], y=FAR[5], u=FAR[7], ws=P, ws_bytes=1 << 40)
    a.update(change)
    assert lib.e8q_lora(ctypes.byref(adapters()), vp(a["x"]), vp(a["slots"]), a["tokens"], vp(a["base"]), vp(a["y"]),
                        vp(a["u"]), vp(a["ws"]), a["ws_bytes"], None) == expect
    assert lib.e8q_lora(None, vp(P), vp(P), 1, None, vp(P), None, vp(P), 1 << 40, None) == 1


@pytest.mark.parametrize("change,expect", [
    (dict(gy=None), 1), (dict(gy=FAR[3] + 8), 1), (dict(x=None), 1), (dict(u=None), 1), (dict(u=FAR[5] + 4), 1),
    (dict(slots=None), 1), (dict(tokens=-1), 1), (dict(tokens=65537), 2), (dict(ga=None), 1), (dict(gb=None), 1),
    (dict(ga=FAR[7] + 2), 1), (dict(gb=FAR[7]), 1), (dict(gx=None), 1), (dict(gx=FAR[10] + 8), 1), (dict(gx0=FAR[9] + 2), 1),
    (dict(ga=FAR[0]), 1), (dict(gb=FAR[1]), 1), (dict(gx=FAR[4]), 1), (dict(gx=FAR[9] + 16), 1), (dict(gx=FAR[7]), 1),
    (dict(ga=FAR[9]), 1), (dict(ws=None), 4), (dict(ws=P + 16), 4), (dict(ws_bytes=1000), 4),
])
def test_lora_backward_refusals(lib, change, expect):
    a = dict(gy=FAR[3], x=FAR[4], u=FAR[5], slots=FAR[6], tokens=5, ga=FAR[7], gb=FAR[8], gx0=FAR[9], gx=FAR[10], ws=P,
             ws_bytes=1 << 40)
    a.update(change)
    assert lib.e8q_lora_backward(ctypes.byref(adapters()), vp(a["gy"]), vp(a["x"]), vp(a["u"]), vp(a["slots"]), a["tokens"],
                                 vp(a["ga"]), vp(a["gb"]), vp(a["gx0"]), vp(a["gx"]), vp(a["ws"]), a["ws_bytes"],
                                 None) == expect


def test_lora_workspace(lib):
    """Holds the grouped order and the partial sums, serves any smaller number
    of tokens (a captured call goes on using it), and the backward pass needs
    more."""
    f = lib.e8q_lora_workspace_bytes
    sizes = list(range(1, 700)) + list(range(700, 9000, 61)) + [65535, 65536]
    for kw in (dict(), dict(rank=128, rows=14336, cols=4096), dict(n=0), dict(n=2048, rows=8, cols=8), dict(n=200, cols=14336),
               dict(n=1, rows=1 << 20, cols=40)):
        a = ctypes.byref(adapters(**kw))
        for backward in (0, 1):
            got = [f(a, t, backward) for t in sizes]
            assert got == sorted(got) and all(b % 256 == 0 for b in got) and got[-1] >= 4 * 65536
        assert all(f(a, t, 1) > f(a, t, 0) >= 4 * t for t in (1, 128, 129, 4096, 65536))
        assert f(a, 65537, 0) == 256 and f(a, -1, 0) == 256 and f(a, 0, 0) == 256
