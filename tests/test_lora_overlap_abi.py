"""The adapters refuse outputs that lie in the adapters' own buffers (CPU:
before any device work; the addresses are never dereferenced)."""
import ctypes

import pytest

from test_lora_abi import FAR, P, adapters, lib, vp  # noqa: F401  (lib: the fixture)

# adapters(): a [4][16][64], b [4][128][16] bf16, scale [4] float32, at FAR[0], FAR[1], FAR[2]
INSIDE = [(FAR[0], 1), (FAR[0] + 4 * 16 * 64 * 2 - 16, 1), (FAR[1], 1), (FAR[1] + 4 * 128 * 16 * 2 - 16, 1), (FAR[2], 1),
          (FAR[0] - 16, 1)]


@pytest.mark.parametrize("at,expect", INSIDE)
def test_forward_outputs_inside_the_adapters(lib, at, expect):  # noqa: F811
    a = ctypes.byref(adapters())
    for y, u in ((at, None), (FAR[5], at)):
        assert lib.e8q_lora(a, vp(FAR[3]), vp(FAR[4]), 5, None, vp(y), vp(u), vp(P), 1 << 40, None) == expect


@pytest.mark.parametrize("at,expect", INSIDE)
def test_backward_outputs_inside_the_adapters(lib, at, expect):  # noqa: F811
    a = ctypes.byref(adapters())
    for ga, gb, gx in ((at, FAR[8], FAR[10]), (FAR[7], at, FAR[10]), (FAR[7], FAR[8], at)):
        assert lib.e8q_lora_backward(a, vp(FAR[3]), vp(FAR[4]), vp(FAR[5]), vp(FAR[6]), 5, vp(ga), vp(gb), None, vp(gx),
                                     vp(P), 1 << 40, None) == expect

    for ga, gb in ((at, FAR[8]), (FAR[7], at)):  # without tokens they are cleared
        assert lib.e8q_lora_backward(a, None, None, None, None, 0, vp(ga), vp(gb), None, None, None, 0, None) == expect


def test_no_adapters_have_no_bytes_to_lie_in(lib):  # noqa: F811
    """n = 0: the addresses are not looked at (the workspace that is refused comes after the overlaps)."""
    a = ctypes.byref(adapters(n=0))
    assert lib.e8q_lora(a, vp(FAR[3]), vp(FAR[4]), 5, None, vp(FAR[0] - 16), None, None, 0, None) == 4
    assert lib.e8q_lora_backward(a, vp(FAR[3]), vp(FAR[4]), vp(FAR[5]), vp(FAR[6]), 5, None, None, None, vp(FAR[2] - 16),
                                 None, 0, None) == 4
