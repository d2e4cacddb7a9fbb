"""Gradients of adapters that hold very many tokens, against float64.

The inputs have one sign, so that what the additions of a long sum lose adds
up.  Bounds as in test_lora_gpu.py, but with a number of additions that does
not grow with the tokens of a CTA: at most 2,048 tokens meet in one
tensor-core accumulator (16 a MMA, high and low part: 256 additions, 16
inside one), and the sums of such units (32 at 65,536 tokens) are added in
fp32.  A result has to lie between the bf16 roundings of value - bound and of
value + bound: rounding keeps the order, so nothing is added for it.
"""
import pytest
import torch

from test_lora_gpu import D_LONG, PART, STEP

pytestmark = pytest.mark.gpu
D = 2048 // 16 * 2 + 16 + 32


def between(got, want, tol, what):
    low, high = (want - tol).bfloat16(), (want + tol).bfloat16()
    bad = ~((got >= low) & (got <= high))
    assert not bad.any(), (what, int(bad.sum()), got.numel(), ((got.double() - want) / want)[bad][:5].tolist())


def summed(a, b):
    """a^T b in float64, a few thousand columns of a at a time."""
    b = b.double()
    return torch.cat([a[:, c:c + 2048].double().t() @ b for c in range(0, a.shape[1], 2048)])


@pytest.mark.parametrize("tokens,cols,rows,rank", [(65536, 8, 38144, 8), (65536, 38144, 8, 8), (20000, 18944, 19200, 40),
                                                   (16384, 19200, 18944, 128), (65536, 520, 512, 16)])
def test_gradients_of_one_adapter_with_every_token(tokens, cols, rows, rank):
    from bit_e8_lattice_b200 import e8q

    g = torch.Generator("cuda").manual_seed(tokens + rank)

    def rand(*shape):
        return (0.5 + torch.rand(shape, device="cuda", generator=g)).bfloat16()

    a, b, x, gy = rand(2, rank, cols), rand(2, rows, rank), rand(tokens, cols), rand(tokens, rows)
    u = 0.5 + torch.rand((tokens, rank), device="cuda", generator=g)
    scale = torch.tensor([0.75, 1.0], device="cuda")
    slots = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    op = e8q.Lora(a, b, scale, tokens)
    ga, gb, _ = op.backward(gy, x, u, slots, need_x=False)
    assert (ga[1] == 0).all() and (gb[1] == 0).all()
    want = 0.75 * summed(gy, u)
    between(gb[0], want, (PART + (D + 2) * STEP) * want, "grad_b")
    v = torch.cat([0.75 * (gy[t:t + 2048].double() @ b[0].double()) for t in range(0, tokens, 2048)])
    want = summed(x, v).t()
    between(ga[0], want, (PART + (D_LONG + D + 2) * STEP) * want, "grad_a")
