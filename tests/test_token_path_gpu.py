"""The row lookup, the 2-bit products, the adapters and the gradients run as a
fine-tuning step runs them: tokens -> rows of an encoded table -> an encoded
projection with adapters beside it -> gradients of the adapters, of the
activations and of the table's latent rows.

Each stage is held to float64 on the stage's own inputs, with the bounds of
the operators' own tests; the chain is also captured into a graph and replayed.
"""
import numpy as np
import pytest
import torch

import oracle
from bit_e8_lattice_b200 import synth
from parity import check_gemv
from test_lora_gpu import backward64, close, forward64
from test_rows_gpu import check_grad, check_lookup, encode, exact_grad, exact_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def e8q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_e8_lattice_b200 import e8q as m

    m.init()
    return m


VOCAB, WIDTH, OUT, RANK, N = 517, 768, 520, 16, 5


class Step:
    """One training step on `tokens` tokens; every buffer is made once."""

    def __init__(self, e8q, tokens, seed=0):
        self.e8q, self.tokens = e8q, tokens
        self.table, self.table_P, self.table_s, _ = encode(e8q, VOCAB, WIDTH, seed=seed + 1)
        self.proj, self.proj_P, self.proj_s, _ = encode(e8q, OUT, WIDTH, seed=seed + 2)
        self.weights = e8q.e8q_decode(self.proj, "original")
        g = torch.Generator("cuda").manual_seed(seed)

        def rand(*shape, std=1.0):
            return (torch.randn(shape, device="cuda", generator=g) * std).bfloat16()

        self.a, self.b = rand(N, RANK, WIDTH, std=WIDTH ** -0.5), rand(N, OUT, RANK, std=0.1)
        self.scale = 0.5 + torch.rand(N, device="cuda", generator=g)
        self.lora = e8q.Lora(self.a, self.b, self.scale, tokens)
        self.product = (e8q.Gemv if tokens <= 64 else e8q.Gemm)(self.proj, tokens)
        self.rows = e8q.RowsBackward(VOCAB, WIDTH, tokens)
        self.ids = torch.empty(tokens, dtype=torch.int64, device="cuda")
        self.slots = torch.empty(tokens, dtype=torch.int32, device="cuda")
        self.grad_y = torch.empty((tokens, OUT), dtype=torch.bfloat16, device="cuda")
        self.x = torch.empty((tokens, WIDTH), dtype=torch.bfloat16, device="cuda")
        self.latent = torch.zeros((VOCAB, WIDTH), dtype=torch.bfloat16, device="cuda")
        self.alpha = WIDTH ** 0.5
        self.draw(seed)

    def draw(self, seed):
        g = torch.Generator("cuda").manual_seed(100 + seed)
        self.ids.copy_(torch.randint(-1, VOCAB, (self.tokens,), device="cuda", generator=g))
        self.slots.copy_(torch.randint(-1, N, (self.tokens,), device="cuda", generator=g))
        self.grad_y.copy_(torch.randn((self.tokens, OUT), device="cuda", generator=g))

    def run(self):
        e8q = self.e8q
        e8q.e8q_decode_rows(self.table, self.ids, alpha=self.alpha, out=self.x)
        self.base = self.product(self.x)
        self.y, self.u = self.lora(self.x, self.slots, base=self.base, keep_u=True)
        self.gx0 = self.grad_y @ self.weights
        self.ga, self.gb, self.gx = self.lora.backward(self.grad_y, self.x, self.u, self.slots, grad_x_base=self.gx0)
        self.rows(self.gx, self.ids, self.latent, alpha=self.alpha)

    def outputs(self):
        return [t.clone() for t in (self.x, self.y, self.u, self.ga, self.gb, self.gx, self.latent)]


@pytest.mark.parametrize("tokens", [1, 37, 64, 128, 200])
def test_fine_tuning_step(e8q, tokens):
    s = Step(e8q, tokens)
    s.run()
    torch.cuda.synchronize()
    if tokens > 64:
        assert s.product.error_word() == 0
    check_lookup(s.x, exact_rows(s.table, s.table_P, s.table_s, "original", 0), s.ids, 0, s.alpha, "original")
    x64 = s.x.double().cpu().numpy()
    live = np.abs(x64).sum(1) > 0  # padding ids give zero rows, whose products have no scale to be held to
    y_ref = oracle.gemv(s.proj_P.reshape(-1, 8), s.proj_s, s.proj.signs.cpu().numpy(), oracle.default_block(WIDTH), x64)
    if live.any():
        check_gemv(s.base[torch.from_numpy(live).cuda()].cpu().view(torch.int16).numpy(), y_ref[live])
    d = dict(a=s.a, b=s.b, scale=s.scale, x=s.x, base=s.base, slots=s.slots, grad_y=s.grad_y, gx0=s.gx0)
    wy, ty, wu, tu = forward64(d)
    close(s.y, wy, ty, "y")
    close(s.u, wu, tu, "u")
    for got, (want, tol), what in zip((s.ga, s.gb, s.gx), backward64(d, s.u), ("grad_a", "grad_b", "grad_x")):
        close(got, want, tol, what)
    want, tol = exact_grad(s.gx, s.ids, VOCAB, 0, s.alpha)
    check_grad(s.latent, want, tol)


@pytest.mark.parametrize("tokens", [1, 200])
def test_fine_tuning_step_in_a_graph(e8q, tokens):
    s = Step(e8q, tokens, seed=3)
    s.run()  # workspaces and tables exist before the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for seed in (5, 6):
        s.draw(seed)
        s.latent.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        replayed = s.outputs()
        other = Step(e8q, tokens, seed=3)
        other.draw(seed)
        other.run()
        torch.cuda.synchronize()
        for a, b in zip(replayed, other.outputs()):
            assert torch.equal(a, b)
