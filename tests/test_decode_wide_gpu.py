"""e8q_decode on rows wider than the fast kernel's tile (14,336 columns)."""
import numpy as np
import pytest
import torch

from bit_e8_lattice_b200 import synth
from parity import check_original_dequant, check_rotated_dequant, gpu_points

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cols,block", [(14336, 2048), (14592, 256), (15872, 512), (16384, 2048)])
def test_decode_rows_up_to_the_widest(cols, block):
    """Every column of the row is decoded, in both bases."""
    from bit_e8_lattice_b200 import e8q

    rows = 3
    w = torch.from_numpy(np.random.default_rng(cols).standard_normal((rows, cols)).astype(np.float32) * 0.02)
    d = synth.signs(1, cols)
    cap = rows * cols // 8
    res = e8q.e8q_project_encode(w.bfloat16().cuda(), torch.from_numpy(d).cuda(), esc_cap=cap, ovf_cap=cap)
    m = res.encoded[0]
    P, *_ = gpu_points(m.idx.cpu().numpy().view(np.uint16).reshape(-1), res.escape_records(), res.overflow_records(), cap)
    scale = m.scale.cpu().numpy()
    for basis, check in (("rotated", check_rotated_dequant), ("original", check_original_dequant)):
        out = torch.full((rows, cols), float("nan"), dtype=torch.bfloat16, device="cuda")
        e8q.e8q_decode(m, basis, out)
        check(out.cpu().view(torch.int16).numpy(), P, scale, d, block, f"{cols} {basis}")
