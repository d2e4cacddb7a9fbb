"""The lookup and its gradient are transposes of one another: for a table with
the rows W,  <g, lookup(ids)> = <G(g, ids), W>  with the same alpha, first row
and ids (outside ones among them), on every way that the gradient orders ids.

Both sides are sums of the same products alpha g W in float64.  With u = 2^-24:
an element of the lookup in fp32 is within 5 u of alpha W, one of W within 5 u,
and G within (m + 3) u alpha sum |g| of its value for a row of m tokens
(test_rows_gpu.py), so the sides differ by at most (m + 13) u of the products'
magnitudes, row by row; 2^-8 of that is allowed for second order.
"""
import pytest
import torch

from test_rows_gpu import U, e8q, encode  # noqa: F401  (e8q: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,ids_dtype", [(1, torch.int64), (100, torch.int32), (3000, torch.int64), (9000, torch.int32)])
@pytest.mark.parametrize("alpha,first", [(1.75, 0), (-64.0, 12345), (0.3, -7)])
def test_lookup_and_gradient_are_transposes(e8q, n, ids_dtype, alpha, first):  # noqa: F811
    rows, cols = 300, 768
    m, *_ = encode(e8q, rows, cols, seed=2)
    g = torch.Generator("cuda").manual_seed(n)
    ids = (torch.randint(-20, rows + 20, (n,), device="cuda", generator=g) + first).to(ids_dtype)
    ids[: n // 3] = first + 5  # a frequent one
    grad = torch.randn((n, cols), device="cuda", generator=g)
    W = e8q.e8q_decode_rows(m, torch.arange(rows, device="cuda"), out_dtype=torch.float32).double()
    x = e8q.e8q_decode_rows(m, ids, alpha=alpha, first_row=first, out_dtype=torch.float32).double()
    G = e8q.e8q_rows_backward(grad, ids, rows, alpha=alpha, first_row=first, latent_dtype=torch.float32).double()
    row = ids.long() - first
    inside = (row >= 0) & (row < rows)
    assert (x[~inside] == 0).all() and inside.any()
    magnitude = abs(alpha) * (grad.double()[inside] * W[row[inside]]).abs().sum(1)
    tokens = torch.bincount(row[inside], minlength=rows)[row[inside]]
    tol = ((tokens + 13) * U * magnitude).sum() * (1 + 2.0 ** -8)
    assert ((grad.double() * x).sum() - (G * W).sum()).abs() <= tol
    # and row by row: a token's part is its own row's
    for r in (5, 0, rows - 1, int(row[inside][-1])):
        at = row == r
        mine = tol if not at.any() else ((at.sum() + 13) * U * abs(alpha) * (grad.double()[at] * W[r]).abs().sum()) * (1 + 2.0 ** -8)
        assert ((grad.double()[at] * x[at]).sum() - (G[r] * W[r]).sum()).abs() <= mine
