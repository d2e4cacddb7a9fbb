"""Lookup of rows of an encoded matrix (e8q_decode_rows) and its gradient
(e8q_rows_backward) on the GPU, against float64.

Tolerances.  u = 2^-24 and 2^-8 are half a step of fp32 and bf16.
Lookup, original basis: the integer transform is exact below 2^24, and
alpha s, sqrt(B), their quotient and the product round once each: 4 u of the
value (5 u allows for second order), and for bf16 another 2^-8.  Rotated
basis: alpha s and the product: 3 u.  Gradient: a sum of m fp32 terms, in any
order, is within (m - 1) u of sum |g|, alpha and the fused add of what is
there round once each: (m + 3) u (alpha sum |g| + |there|), and 2^-8 for bf16.
"""
import numpy as np
import pytest
import torch

import oracle
from bit_e8_lattice_b200 import synth
from parity import gpu_points

pytestmark = pytest.mark.gpu
U, HALF = 2.0 ** -24, {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def e8q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_e8_lattice_b200 import e8q as m

    m.init()
    return m


def encode(e8q, rows, cols, block=0, kappa=1.0, seed=0, extra=0):
    """An encoded matrix, its lattice points [rows][cols] (doubled) and the
    stored scales; with `extra`, the second matrix of one encode call (its
    records and group ids begin behind the first one's)."""
    rng = np.random.default_rng([seed, rows, cols])
    shapes = ([(extra, 64)] if extra else []) + [(rows, cols)]
    ws = [torch.from_numpy(rng.standard_normal(s).astype(np.float32) * 0.02).bfloat16().cuda() for s in shapes]
    ss = [torch.from_numpy(synth.signs(seed, s[1], i)).cuda() for i, s in enumerate(shapes)]
    cap = sum(s[0] * s[1] // 8 for s in shapes) + 64
    enc = e8q.Encoder(shapes, ss, torch.bfloat16, [0] * (len(shapes) - 1) + [block], kappa, esc_cap=cap, ovf_cap=cap)
    res = enc(ws)
    torch.cuda.synchronize()
    assert res.read_counters()["n_dropped"] == 0
    m = res.encoded[-1]
    P, *_ = gpu_points(m.idx.cpu().numpy().view(np.uint16).reshape(-1), res.escape_records(), res.overflow_records(),
                       rows * cols // 8, m.group_base)
    return m, P.reshape(rows, cols), m.scale.cpu().numpy().astype(np.float64), res


def exact_rows(m, P, scale, basis, block):
    if basis == "rotated":
        return scale[:, None] * P / 2.0
    B = oracle.default_block(m.cols) if block == 0 else block
    return oracle.dequant(P, scale, m.signs.cpu().numpy(), B, "original")[1]


def check_lookup(out, rows64, ids, first, alpha, basis, label=""):
    ids = ids.cpu().numpy().astype(object).reshape(-1) - first
    want = np.zeros((len(ids), rows64.shape[1]))
    for t, r in enumerate(ids):
        if 0 <= r < rows64.shape[0]:
            want[t] = np.float64(np.float32(alpha)) * rows64[int(r)]
    got = out.double().cpu().numpy().reshape(want.shape)
    tol = (HALF[out.dtype] + (5 if basis == "original" else 3) * U) * np.abs(want)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (label, int(bad.sum()), np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])


SHAPES = [(5, 8, 0), (7, 24, 0), (9, 40, 1), (6, 96, 16), (11, 64, 8), (13, 256, 0), (33, 768, 0), (5, 1000, 0),
          (17, 2048, 1024), (9, 2048, 0), (10, 2304, 0), (12, 4096, 512), (19, 4096, 0), (3, 14336, 0), (3, 16384, 0)]


@pytest.mark.parametrize("basis", ["original", "rotated"])
@pytest.mark.parametrize("rows,cols,block", SHAPES)
def test_lookup_matches_decode_and_float64(e8q, rows, cols, block, basis):
    """Every block size and odd widths: alpha = 1 in bf16 is e8q_decode's row
    bit for bit; a scaled lookup in both types is within its roundings."""
    m, P, scale, _ = encode(e8q, rows, cols, block, extra=3)
    full = e8q.e8q_decode(m, basis)
    rng = np.random.default_rng(cols)
    ids = torch.from_numpy(np.concatenate([rng.integers(0, rows, 2 * rows + 1), [-1, rows, 2 ** 31 - 1, -2 ** 31]])).int().cuda()
    out = e8q.e8q_decode_rows(m, ids, basis)
    ok = (ids >= 0) & (ids < rows)
    want = torch.where(ok[:, None], full[ids.clamp(0, rows - 1).long()], torch.zeros_like(full[:1]))
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    rows64 = exact_rows(m, P, scale, basis, block)
    for dtype in (torch.bfloat16, torch.float32):
        out = e8q.e8q_decode_rows(m, ids, basis, alpha=0.3, out_dtype=dtype)
        check_lookup(out, rows64, ids, 0, 0.3, basis, f"{rows}x{cols}/{block} {dtype}")


@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 31, 127, 1000, 6001])
def test_lookup_batch_sizes(e8q, n):
    """One token to more windows than the GPU holds at once."""
    m, P, scale, _ = encode(e8q, 61, 4096)
    ids = torch.from_numpy(np.random.default_rng(n).integers(-1, 62, n)).cuda()
    full = e8q.e8q_decode(m, "original")
    want = torch.where(((ids >= 0) & (ids < 61))[:, None], full[ids.clamp(0, 60)], torch.zeros_like(full[:1]))
    assert torch.equal(e8q.e8q_decode_rows(m, ids).view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("kappa,block", [(0.45, 0), (1.5, 0), (3.0, 256), (50.0, 0), (50.0, 1), (50.0, 8), (200.0, 64)])
@pytest.mark.parametrize("cols", [256, 2048, 4096])
def test_lookup_far_points(e8q, kappa, block, cols):
    """From rows without records to rows in which every group is an overflow
    record with coordinates in the hundreds (beyond f16's exact sums)."""
    m, P, scale, _ = encode(e8q, 9, cols, block, kappa, seed=3)
    if kappa == 200.0:
        assert np.abs(P).max() > 512
    ids = torch.tensor([3, 8, 0, 3, -5, 7], device="cuda")
    for basis in ("original", "rotated"):
        rows64 = exact_rows(m, P, scale, basis, block)
        for dtype in (torch.bfloat16, torch.float32):
            check_lookup(e8q.e8q_decode_rows(m, ids, basis, alpha=-2.5, out_dtype=dtype), rows64, ids, 0, -2.5, basis)
        full = e8q.e8q_decode(m, basis)[ids.clamp(min=0)]
        full[4] = 0
        assert torch.equal(e8q.e8q_decode_rows(m, ids, basis).view(torch.int16), full.view(torch.int16))


def test_lookup_mixed_near_and_far_points(e8q):
    """A given scale that is 30 times too small in some rows: near and far
    overflow points in one window."""
    rows, cols = 8, 4096
    rng = np.random.default_rng(7)
    w = rng.standard_normal((rows, cols)) * 0.02
    w[:, ::97] *= 40
    wt = torch.from_numpy(w.astype(np.float32)).bfloat16().cuda()
    cap = rows * cols // 8
    res = e8q.e8q_project_encode(wt, torch.from_numpy(synth.signs(1, cols)).cuda(), rht_block=8, esc_cap=cap, ovf_cap=cap)
    m = res.encoded[0]
    P, *_ = gpu_points(m.idx.cpu().numpy().view(np.uint16).reshape(-1), res.escape_records(), res.overflow_records(),
                       cap, 0)
    s = np.abs(P).reshape(-1, 8).sum(1)
    assert (s > 64).any() and ((s > 30) & (s <= 64)).any()
    for basis in ("original", "rotated"):
        rows64 = exact_rows(m, P.reshape(rows, cols), m.scale.cpu().numpy().astype(np.float64), basis, 8)
        ids = torch.arange(rows, device="cuda")
        check_lookup(e8q.e8q_decode_rows(m, ids, basis, out_dtype=torch.float32), rows64, ids, 0, 1.0, basis)


def test_lookup_of_shards_adds_up_and_offsets_do_not_wrap(e8q):
    m, P, scale, _ = encode(e8q, 40, 768)
    whole = e8q.Encoded(m.idx, m.scale, m.signs, m.esc, m.esc_row_ptr, m.ovf, m.ovf_row_ptr, 40, 768, m.group_base, 0,
                        m.esc_count, m.ovf_count)
    g = 768 // 8
    top = e8q.Encoded(m.idx[:15], m.scale[:15], m.signs, m.esc, m.esc_row_ptr[:16], m.ovf, m.ovf_row_ptr[:16], 15, 768,
                      m.group_base, 0, m.esc_count, m.ovf_count)
    low = e8q.Encoded(m.idx[15:], m.scale[15:], m.signs, m.esc, m.esc_row_ptr[15:], m.ovf, m.ovf_row_ptr[15:], 25, 768,
                      m.group_base + 15 * g, 0, m.esc_count, m.ovf_count)
    for base in (0, 2 ** 40, -2 ** 62):
        ids = torch.randint(-1, 41, (7, 30), device="cuda") + base
        a = e8q.e8q_decode_rows(whole, ids, first_row=base)
        b = e8q.e8q_decode_rows(top, ids, first_row=base) + e8q.e8q_decode_rows(low, ids, first_row=base + 15)
        assert a.shape == (7, 30, 768) and torch.equal(a, b)
    far = torch.tensor([2 ** 63 - 1, -2 ** 63, 0, 39], device="cuda")
    out = e8q.e8q_decode_rows(whole, far, first_row=-2 ** 63)
    assert (out[[0, 2, 3]] == 0).all() and torch.equal(out[1], e8q.e8q_decode(whole, "original")[0])


def test_lookup_without_records_rows_or_ids(e8q):
    """No record arrays, an empty matrix, no ids."""
    m, *_ = encode(e8q, 4, 64, kappa=0.3)
    bare = e8q.Encoded(m.idx, m.scale, m.signs, None, None, None, None, 4, 64, 0, 0)
    ids = torch.tensor([2, 2, 9], device="cuda")
    want = e8q.e8q_decode(bare, "original")[[2, 2, 0]]
    want[2] = 0
    assert torch.equal(e8q.e8q_decode_rows(bare, ids), want)
    empty = torch.zeros(0, dtype=torch.uint8, device="cuda")
    ptr = torch.zeros(5, dtype=torch.int64, device="cuda")
    bare = e8q.Encoded(m.idx, m.scale, m.signs, empty, ptr, empty, ptr, 4, 64, 0, 0)
    assert torch.equal(e8q.e8q_decode_rows(bare, ids), want)
    none = e8q.Encoded(m.idx[:0], m.scale[:0], m.signs, None, None, None, None, 0, 64, 0, 0)
    assert (e8q.e8q_decode_rows(none, ids, out=torch.ones((3, 64), device="cuda")) == 0).all()
    assert e8q.e8q_decode_rows(m, ids[:0]).shape == (0, 64)


def test_lookup_with_malformed_records(e8q):
    """Row pointers that are negative, past the records or descending, groups
    of other rows and roots that do not exist: those records are left out,
    and rows with sound pointers read as before."""
    rows, cols = 24, 2048
    m, *_ = encode(e8q, rows, cols)
    want = e8q.e8q_decode(m, "original")
    n_esc, n_ovf = int(m.esc_row_ptr[-1]), int(m.ovf_row_ptr[-1])
    bare = e8q.Encoded(m.idx, m.scale, m.signs, None, None, None, None, rows, cols, 0, 0)
    plain = e8q.e8q_decode(bare, "original")  # no record at all
    ids = torch.arange(rows, device="cuda")
    for ends in ((-5, -1), (2 ** 62, 2 ** 62 + 9), (n_esc, n_esc + 10 ** 9), (7, 3), (2 ** 32 + 4, 2 ** 32 + 1)):
        erp, orp = m.esc_row_ptr.clone(), m.ovf_row_ptr.clone()
        erp[8], erp[9] = ends
        orp[8], orp[9] = ends
        bad = e8q.Encoded(m.idx, m.scale, m.signs, m.esc[: 8 * n_esc], erp, m.ovf[: 20 * n_ovf], orp, rows, cols, 0, 0,
                          n_esc, n_ovf)
        out = e8q.e8q_decode_rows(bad, ids)
        assert torch.equal(out[:7], want[:7]) and torch.equal(out[10:], want[10:])
        assert torch.equal(out[8], plain[8])
    esc = m.esc[: 8 * n_esc].clone().view(torch.int32).view(-1, 2)
    ovf = m.ovf[: 20 * n_ovf].clone().view(torch.int32).view(-1, 5)
    esc[0::2, 0] = -1                 # a group that no row has
    esc[1::2, 1] |= 0xFF << 16        # root 255
    ovf[:, 0] += cols // 8            # the next row's group
    bad = e8q.Encoded(m.idx, m.scale, m.signs, esc.view(torch.uint8).view(-1), m.esc_row_ptr, ovf.view(torch.uint8).view(-1),
                      m.ovf_row_ptr, rows, cols, 0, 0, n_esc, n_ovf)
    assert torch.equal(e8q.e8q_decode_rows(bad, ids), plain)


def test_lookup_writes_its_rows_only(e8q):
    m, *_ = encode(e8q, 10, 96)
    buf = torch.full((12, 96), 7.0, device="cuda", dtype=torch.bfloat16)
    e8q.e8q_decode_rows(m, torch.arange(8, device="cuda"), out=buf[2:10])
    assert (buf[:2] == 7).all() and (buf[10:] == 7).all()
    assert torch.equal(buf[2:10], e8q.e8q_decode(m, "original")[:8])


# ------------------------------------------------------------------ gradient
def exact_grad(grad, ids, rows, first, alpha, there=None):
    """(value, tolerance without the output's own rounding)."""
    ids = [int(i) - first for i in ids.reshape(-1).cpu().tolist()]
    g = grad.double().cpu().numpy().reshape(len(ids), -1)
    s, a, m = np.zeros((rows, g.shape[1])), np.zeros((rows, g.shape[1])), np.zeros((rows, 1))
    for t, r in enumerate(ids):
        if 0 <= r < rows:
            s[r] += g[t]
            a[r] += np.abs(g[t])
            m[r] += 1
    al = np.float64(np.float32(alpha))
    base = 0.0 if there is None else there.double().cpu().numpy()
    return al * s + base, (m + 3) * U * (abs(al) * a + np.abs(base))


def check_grad(got, want, tol):
    err = np.abs(got.double().cpu().numpy() - want)
    bad = ~(err <= tol * (1 + 2.0 ** -8) + HALF[got.dtype] * np.abs(want))
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3])


@pytest.mark.parametrize("gd,ld", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("n,rows,cols", [(1, 1, 8), (1, 70, 2048), (2, 3, 1032), (37, 5, 64), (128, 1000, 768),
                                         (129, 40, 24), (130, 7, 4096), (700, 3, 1000), (2000, 513, 96), (5000, 20, 40),
                                         (8192, 300, 16), (8193, 300, 16), (9000, 1, 2048), (20000, 70000, 8)])
def test_gradient_matches_float64(e8q, n, rows, cols, gd, ld):
    """Every path (direct, ranked, radix with one to two digits), runs from
    one token to all tokens on one row, rows without a token, ids outside."""
    rng = np.random.default_rng([n, rows, cols])
    first = 11
    ids = first + np.minimum(np.floor(rng.exponential(max(rows / 6, 0.3), n)), rows).astype(np.int64)
    ids[rng.random(n) < 0.05] = -1
    ids = torch.from_numpy(ids).cuda()
    grad = torch.randn((n, cols), device="cuda", generator=torch.Generator("cuda").manual_seed(n)).to(gd)
    op = e8q.RowsBackward(rows, cols, n, gd, ld)
    out = torch.full((rows, cols), float("nan"), device="cuda", dtype=ld)  # every row has to be written
    got = op(grad, ids, out, alpha=0.7, first_row=first).clone()
    want, tol = exact_grad(grad, ids, rows, first, 0.7)
    check_grad(got, want, tol)
    assert torch.equal(got, op(grad, ids.int(), out, alpha=0.7, first_row=first))  # the same bits again, int32 ids
    there = torch.randn((rows, cols), device="cuda").to(ld)
    acc = there.clone()
    op(grad, ids, acc, alpha=0.7, first_row=first, accumulate=True)
    want, tol = exact_grad(grad, ids, rows, first, 0.7, there)
    check_grad(acc, want, tol)
    touched = torch.zeros(rows, dtype=torch.bool, device="cuda")
    inside = (ids >= first) & (ids < first + rows)
    touched[(ids[inside] - first)] = True
    assert torch.equal(acc[~touched], there[~touched])


@pytest.mark.parametrize("n", [100, 128, 129, 1000, 8192, 8200, 40000, 300000])
def test_gradient_of_one_row_and_of_distinct_rows(e8q, n):
    """All tokens on one row (a padding id), and every row exactly once."""
    cols = 264
    grad = torch.randn((n, cols), device="cuda", generator=torch.Generator("cuda").manual_seed(n))
    for ids in (torch.full((n,), 5, device="cuda"), torch.randperm(n, device="cuda"),
                torch.full((n,), -1, device="cuda")):
        rows = max(n, 6)
        got = e8q.e8q_rows_backward(grad, ids, rows, latent_dtype=torch.float32)
        s = torch.zeros((rows + 1, cols), device="cuda", dtype=torch.float64)
        a = torch.zeros_like(s)
        at = torch.where(ids < 0, rows, ids)
        s.index_add_(0, at, grad.double())
        a.index_add_(0, at, grad.double().abs())
        m = torch.bincount(at, minlength=rows + 1)[:, None]
        assert ((got.double() - s[:-1]).abs() <= ((m + 3) * U * a)[:-1]).all()


def test_gradient_radix_sort_of_wide_ids(e8q):
    """Three digits of row ids (2^22 rows), ids at both ends of the table."""
    rows, cols, n = (1 << 22) + 3, 8, 30001
    g = torch.Generator("cuda").manual_seed(1)
    ids = torch.randint(0, rows, (n,), device="cuda", generator=g)
    ids[:5] = torch.tensor([0, rows - 1, rows, -1, 0], device="cuda")
    grad = torch.randint(-8, 9, (n, cols), device="cuda", generator=g).bfloat16()  # exact sums
    got = e8q.e8q_rows_backward(grad, ids, rows, latent_dtype=torch.float32)
    want = torch.zeros((rows + 1, cols), device="cuda")
    want.index_add_(0, torch.where(ids < 0, rows, ids.clamp(max=rows)), grad.float())
    assert torch.equal(got, want[:-1])


def test_gradient_is_the_lookups_transpose(e8q):
    """<G, W> = <g, lookup(W)> for the rows of a dense table (here: one-hot
    rows), and against differences of the loss sum(g * alpha * W[ids])."""
    rows, cols, n, alpha = 12, 16, 50, 1.75
    g = torch.Generator("cuda").manual_seed(3)
    ids = torch.randint(-1, rows + 1, (n,), device="cuda", generator=g)
    grad = torch.randn((n, cols), device="cuda", generator=g)
    W = torch.randn((rows, cols), device="cuda", generator=g, dtype=torch.float64)

    def loss(w):
        ok = ((ids >= 0) & (ids < rows))[:, None]
        return (torch.where(ok, w[ids.clamp(0, rows - 1)], 0.0) * alpha * grad.double()).sum()

    G = e8q.e8q_rows_backward(grad, ids, rows, alpha=alpha, latent_dtype=torch.float32).double()
    for r, c in ((0, 0), (5, 3), (11, 15)):
        e = torch.zeros_like(W)
        e[r, c] = 0.5
        diff = (loss(W + e) - loss(W - e)).item()  # the loss is linear: exact but for float64
        assert abs(diff - G[r, c].item()) <= 60 * U * abs(alpha) * grad[ids == r, c].abs().sum().item() + 1e-12


def test_gradient_nan_and_inf_stay_in_their_rows(e8q):
    n, rows, cols = 600, 9, 64
    ids = torch.arange(n, device="cuda") % (rows + 2) - 1
    grad = torch.ones((n, cols), device="cuda")
    grad[ids == 3] = float("nan")
    grad[ids == -1] = float("nan")
    grad[ids == rows] = float("inf")
    grad[(ids == 5).nonzero()[0]] = float("inf")
    got = e8q.e8q_rows_backward(grad, ids, rows, latent_dtype=torch.float32)
    assert got[3].isnan().all() and got[5].isinf().all()
    keep = [0, 1, 2, 4, 6, 7, 8]
    assert torch.equal(got[keep], torch.stack([(ids == r).sum().float().expand(cols) for r in keep]))


def test_gradient_no_ids(e8q):
    out = torch.ones((5, 16), device="cuda", dtype=torch.bfloat16)
    ids = torch.zeros(0, dtype=torch.int64, device="cuda")
    grad = torch.zeros((0, 16), device="cuda", dtype=torch.bfloat16)
    op = e8q.RowsBackward(5, 16, 0)
    assert (op(grad, ids, out.clone(), accumulate=True) == 1).all()
    assert (op(grad, ids, out) == 0).all()


def test_rows_operators_on_other_streams_and_in_graphs(e8q):
    """On a side stream, and captured once and replayed on new inputs."""
    m, *_ = encode(e8q, 50, 768)
    ids = torch.randint(0, 50, (300,), device="cuda")
    grad = torch.randn((300, 768), device="cuda").bfloat16()
    want, wantg = e8q.e8q_decode_rows(m, ids), e8q.e8q_rows_backward(grad, ids, 50)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = e8q.e8q_decode_rows(m, ids, stream=side)
    b = e8q.e8q_rows_backward(grad, ids, 50, stream=side)
    side.synchronize()
    assert torch.equal(a, want) and torch.equal(b, wantg)
    op = e8q.RowsBackward(50, 768, 300)
    out, lat = torch.empty_like(want), torch.empty_like(wantg)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        e8q.e8q_decode_rows(m, ids, out=out)
        op(grad, ids, lat)
    for seed in range(3):
        ids.copy_(torch.randint(-1, 51, (300,), device="cuda"))
        grad.copy_(torch.randn((300, 768), device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, e8q.e8q_decode_rows(m, ids))
        assert torch.equal(lat, e8q.e8q_rows_backward(grad, ids, 50))


def test_rows_past_32_bit_offsets(e8q):
    """More than 2^31 elements on the tokens' side (4.4 GB of bf16)."""
    m, *_ = encode(e8q, 100, 4096)
    n = 2 ** 31 // 4096 + 1000
    ids = torch.arange(n, device="cuda") % 100
    out = e8q.e8q_decode_rows(m, ids)
    want = e8q.e8q_decode(m, "original")
    assert torch.equal(out[-1500:], want[ids[-1500:]]) and torch.equal(out[:100], want)
    out.fill_(1)
    out[-1] = 3
    G = e8q.e8q_rows_backward(out, ids, 100, latent_dtype=torch.float32)  # whole numbers: exact
    want = torch.bincount(ids, minlength=100).float()
    want[ids[-1]] += 2
    assert torch.equal(G, want[:, None].expand(100, 4096))


def test_rows_backward_device_argument(e8q):
    """A device without an index is the current one."""
    op = e8q.RowsBackward(4, 8, 2, device="cuda")
    ids = torch.tensor([3, 3], device="cuda")
    got = op(torch.ones((2, 8), device="cuda").bfloat16(), ids)
    assert (got[3] == 2).all() and (got[:3] == 0).all()
    for bad in (dict(rows=-1), dict(cols=0), dict(max_ids=-1), dict(grad_dtype=torch.float16)):
        with pytest.raises(e8q.E8qError):
            e8q.RowsBackward(**{**dict(rows=4, cols=8, max_ids=2), **bad})


def test_rows_refuse_bad_tensors(e8q):
    m, *_ = encode(e8q, 6, 64)
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    for bad in (dict(ids=ids.cpu()), dict(ids=ids.float()), dict(ids=ids.expand(3, 4).t()), dict(basis="none"),
                dict(out_dtype=torch.float16), dict(alpha=float("inf")),
                dict(out=torch.empty((4, 72), device="cuda")), dict(out=torch.empty((4, 64), device="cuda").half()),
                dict(out=torch.empty((4, 128), device="cuda")[:, :64]),
                dict(out=torch.empty(4 * 64 + 1, device="cuda")[1:].view(4, 64))):
        with pytest.raises(e8q.E8qError):
            e8q.e8q_decode_rows(**{**dict(m=m, ids=ids), **bad})
    op = e8q.RowsBackward(6, 64, 4)
    grad, lat = torch.zeros((4, 64), device="cuda").bfloat16(), torch.zeros((6, 64), device="cuda").bfloat16()
    for bad in (dict(grad_out=grad.float()), dict(grad_out=grad[:3]), dict(ids=ids.short()), dict(grad_latent=lat[:5]),
                dict(grad_latent=lat.float()), dict(grad_latent=None, accumulate=True), dict(alpha=float("nan")),
                dict(grad_out=torch.zeros((8, 64), device="cuda").bfloat16(), ids=torch.zeros(8, dtype=torch.int64, device="cuda")),
                dict(grad_out=lat[:4])):
        with pytest.raises(e8q.E8qError):
            op(**{**dict(grad_out=grad, ids=ids, grad_latent=lat), **bad})
