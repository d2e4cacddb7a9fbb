"""Low-rank adapters (e8q_lora, e8q_lora_backward) on the GPU against float64.

Tolerances.  Products of bf16 values are exact in fp32.  A tensor-core sum is
taken to lose at most one fp32 step, 2^-23, of the sum of magnitudes at
each addition (a truncating adder's bound); D below counts the additions
on the longest path: the MMAs of one warp's range, 16 inside an MMA, and
the joins of warps, splits and units.  A factor in two bf16 parts is off by
half a step of the low part, 2^-8 2^-8 = 2^-16 of its value.  The result rounds
to bf16 once: 2^-8 of its value.  Errors of a factor pass on through the
magnitudes of what it multiplies.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
STEP, PART, HALF = 2.0 ** -23, 2.0 ** -16, 2.0 ** -8
D_LONG = 64 + 16 + 8 + 70  # k_lr_down: 4,096 columns over 4 warps of 16-column MMAs at most; warps; splits


@pytest.fixture(scope="module")
def e8q():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from bit_e8_lattice_b200 import e8q as m

    m.init()
    return m


def make(tokens, cols, rows, rank, n, seed=0, slots=None):
    g = torch.Generator("cuda").manual_seed(seed * 1000 + tokens)

    def rand(*shape, std=1.0):
        return (torch.randn(shape, device="cuda", generator=g) * std).bfloat16()

    d = dict(a=rand(n, rank, cols, std=cols ** -0.5), b=rand(n, rows, rank, std=rank ** -0.5), x=rand(tokens, cols),
             base=rand(tokens, rows), scale=0.5 + torch.rand(n, device="cuda", generator=g),
             grad_y=rand(tokens, rows), gx0=rand(tokens, cols))
    if slots is None:
        slots = torch.randint(-1, n + 1, (tokens,), device="cuda", generator=g)
    d["slots"] = slots.to(torch.int32)
    return d


def forward64(d, base=True):
    """y, u and their tolerances."""
    T, n = d["x"].shape[0], d["a"].shape[0]
    y = d["base"].double() if base else torch.zeros_like(d["base"].double())
    ytol = torch.zeros_like(y)
    u = torch.zeros((T, d["a"].shape[1]), dtype=torch.float64, device="cuda")
    utol = torch.zeros_like(u)
    R = u.shape[1]
    for i in range(n):
        t = (d["slots"] == i).nonzero()[:, 0]
        if not len(t):
            continue
        A, B, x, s = d["a"][i].double(), d["b"][i].double(), d["x"][t].double(), d["scale"][i].double()
        u[t] = x @ A.t()
        utol[t] = D_LONG * STEP * (x.abs() @ A.abs().t())
        y[t] += s * (u[t] @ B.t())
        ytol[t] = s * (utol[t] + (PART + (R // 8 + 18 + 2) * STEP) * u[t].abs()) @ B.abs().t()
    return y, ytol + HALF * y.abs() + STEP * y.abs(), u, utol


def backward64(d, u):
    n, R = d["a"].shape[0], d["a"].shape[1]
    ga, gb, gx = d["a"].double() * 0, d["b"].double() * 0, d["gx0"].double()
    ta, tb, tx = torch.zeros_like(ga), torch.zeros_like(gb), torch.zeros_like(gx)
    for i in range(n):
        t = (d["slots"] == i).nonzero()[:, 0]
        if not len(t):
            continue
        A, B, x, s = d["a"][i].double(), d["b"][i].double(), d["x"][t].double(), d["scale"][i].double()
        gy, ui = d["grad_y"][t].double(), u[t].double()
        D = len(t) / 8 + 16 + 80  # hi and lo MMAs over the tokens, joins of units
        v = s * (gy @ B)
        vtol = s * D_LONG * STEP * (gy.abs() @ B.abs()) + (PART + 2 * STEP) * v.abs()
        ga[i] = v.t() @ x
        ta[i] = vtol.t() @ x.abs() + D * STEP * (v.abs().t() @ x.abs())
        gb[i] = s * (gy.t() @ ui)
        tb[i] = s * (PART + (D + 2) * STEP) * (gy.abs().t() @ ui.abs())
        gx[t] += v @ A
        tx[t] = (vtol + (R // 8 + 20) * STEP * v.abs()) @ A.abs()
    return [(w, tol + (HALF + STEP) * w.abs()) for w, tol in ((ga, ta), (gb, tb), (gx, tx))]


def close(got, want, tol, what):
    err = (got.double() - want).abs()
    bad = ~(err <= tol + 1e-30)
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[:3].tolist(), (err / (tol + 1e-30)).max().item())


SHAPES = [(1, 8, 8, 8, 1), (1, 4096, 4096, 16, 32), (2, 40, 264, 8, 3), (7, 96, 16, 24, 2), (8, 264, 1000, 32, 5),
          (9, 1000, 96, 64, 4), (33, 2048, 768, 16, 33), (64, 520, 136, 128, 64), (65, 136, 520, 40, 1),
          (128, 768, 2048, 16, 7), (129, 768, 2048, 16, 7), (130, 24, 40, 128, 2), (300, 4104, 72, 72, 3),
          (500, 8, 4104, 8, 40), (1000, 296, 328, 48, 2), (1500, 256, 264, 112, 1), (2100, 64, 48, 16, 2048),
          (4099, 520, 512, 32, 6), (64, 14336, 512, 16, 64), (70, 512, 14336, 64, 3)]


@pytest.mark.parametrize("tokens,cols,rows,rank,n", SHAPES)
def test_adapters_match_float64(e8q, tokens, cols, rows, rank, n):
    """Forward and backward: ranks 8 to 128, odd widths, one token to many,
    one adapter to thousands, tokens without one."""
    d = make(tokens, cols, rows, rank, n)
    op = e8q.Lora(d["a"], d["b"], d["scale"], tokens)
    y, u = op(d["x"], d["slots"], base=d["base"], keep_u=True)
    y, u = y.clone(), u.clone()
    wy, ty, wu, tu = forward64(d)
    close(u, wu, tu, "u")
    close(y, wy, ty, "y")
    assert torch.equal(y, op(d["x"], d["slots"], base=d["base"]))  # the same bits, without u
    y0 = op(d["x"], d["slots"]).clone()
    close(y0, *forward64(d, base=False)[:2], "y without base")
    inplace = d["base"].clone()
    assert torch.equal(op(d["x"], d["slots"], base=inplace, out=inplace), y)
    ga, gb, gx = (t.clone() for t in op.backward(d["grad_y"], d["x"], u, d["slots"], grad_x_base=d["gx0"]))
    for got, (want, tol), what in zip((ga, gb, gx), backward64(d, u), ("grad_a", "grad_b", "grad_x")):
        close(got, want, tol, what)
    again = op.backward(d["grad_y"], d["x"], u, d["slots"], need_x=False)
    assert torch.equal(again[0], ga) and torch.equal(again[1], gb) and again[2] is None
    gx2 = d["gx0"].clone()
    op.backward(d["grad_y"], d["x"], u, d["slots"], grad_x_base=gx2, grad_x=gx2)
    assert torch.equal(gx2, gx)


@pytest.mark.parametrize("tokens", [5, 64, 128, 200, 1000])
@pytest.mark.parametrize("kind", ["one", "none", "runs", "last", "outside"])
def test_adapters_slot_patterns(e8q, tokens, kind):
    """All tokens on one adapter, on none, in runs, on the last only, and
    slots far outside the range."""
    n, cols, rows, rank = 6, 200, 264, 16
    t = torch.arange(tokens, device="cuda")
    slots = dict(one=t * 0 + 3, none=t * 0 - 1, runs=(t // 17) % n, last=t * 0 + n - 1,
                 outside=torch.where(t % 3 == 0, t % n, torch.where(t % 3 == 1, t * 0 + n, t * 0 - 2 ** 31)))[kind]
    d = make(tokens, cols, rows, rank, n, slots=slots)
    op = e8q.Lora(d["a"], d["b"], d["scale"], tokens)
    y, u = op(d["x"], d["slots"], base=d["base"], keep_u=True)
    wy, ty, wu, tu = forward64(d)
    close(y, wy, ty, "y")
    close(u, wu, tu, "u")
    free = (d["slots"] < 0) | (d["slots"] >= n)
    assert torch.equal(y[free], d["base"][free]) and (u[free] == 0).all()
    outs = op.backward(d["grad_y"], d["x"], u, d["slots"], grad_x_base=d["gx0"])
    for got, (want, tol), what in zip(outs, backward64(d, u), ("grad_a", "grad_b", "grad_x")):
        close(got, want, tol, what)
    assert torch.equal(outs[2][free], d["gx0"][free])


def test_adapters_do_not_mix_tokens(e8q):
    """A token's result does not depend on its neighbours: NaN and infinities
    stay in their own tokens (forward) and adapters (backward)."""
    for tokens in (40, 300):
        n, cols, rows, rank = 4, 264, 136, 24
        d = make(tokens, cols, rows, rank, n, seed=5)
        op = e8q.Lora(d["a"], d["b"], d["scale"], tokens)
        y, u = (t.clone() for t in op(d["x"], d["slots"], base=d["base"], keep_u=True))
        ga, gb, gx = (t.clone() for t in op.backward(d["grad_y"], d["x"], u, d["slots"], grad_x_base=d["gx0"]))
        bad = {k: v.clone() for k, v in d.items()}
        ill = (d["slots"] == 1).nonzero()[::2, 0]
        free = ((d["slots"] < 0) | (d["slots"] >= n)).nonzero()[:, 0]
        bad["x"][ill] = float("nan")
        bad["x"][free] = float("inf")
        bad["grad_y"][ill[0]] = float("inf")
        bad["grad_y"][free] = float("nan")
        y2, u2 = (t.clone() for t in op(bad["x"], d["slots"], base=d["base"], keep_u=True))
        well = torch.ones(tokens, dtype=torch.bool, device="cuda")
        well[ill] = False
        assert torch.equal(y2[well], y[well]) and torch.equal(u2[well], u[well]) and y2[ill].isnan().all()
        ga2, gb2, gx2 = op.backward(bad["grad_y"], bad["x"], u2, d["slots"], grad_x_base=d["gx0"])
        keep = [0, 2, 3]
        assert torch.equal(ga2[keep], ga[keep]) and torch.equal(gb2[keep], gb[keep])
        well[ill[0]] = False
        ok = well.clone()
        ok[ill[1:]] = True  # their grad_y is finite
        assert torch.equal(gx2[ok], gx[ok])
        assert not ga2[1].isfinite().all() and not gb2[1].isfinite().all()


def test_adapters_permuted_tokens_give_the_same_rows(e8q):
    d = make(200, 264, 136, 16, 9, seed=2)
    op = e8q.Lora(d["a"], d["b"], d["scale"], 200)
    y, u = (t.clone() for t in op(d["x"], d["slots"], base=d["base"], keep_u=True))
    p = torch.randperm(200, device="cuda")
    y2, u2 = op(d["x"][p], d["slots"][p], base=d["base"][p], keep_u=True)
    assert torch.equal(u2, u[p]) and torch.equal(y2, y[p])


def test_adapter_gradients_against_differences(e8q):
    """The loss sum(g * y) with y in float64, differentiated by central
    differences (y is linear in A, in B and in x), against the kernels."""
    d = make(90, 64, 72, 8, 3, seed=4)
    op = e8q.Lora(d["a"], d["b"], d["scale"], 90)
    _, u = op(d["x"], d["slots"], base=d["base"], keep_u=True)
    got = dict(zip(("a", "b", "x"), op.backward(d["grad_y"], d["x"], u, d["slots"])))
    f = {k: d[k].double() for k in ("a", "b", "x")}
    sl = d["slots"].long()

    def loss(v):
        total = 0.0
        for i in range(3):
            t = (sl == i).nonzero()[:, 0]
            total = total + d["scale"][i].double() * ((v["x"][t] @ v["a"][i].t() @ v["b"][i].t()) * d["grad_y"][t].double()).sum()
        return total

    want = backward64(dict(d, gx0=torch.zeros_like(d["x"])), u)
    for name, at, (_, tol) in (("a", (1, 3, 5), want[0]), ("a", (2, 7, 63), want[0]), ("b", (0, 71, 2), want[1]),
                               ("x", (11, 40), want[2])):
        e = {k: v.clone() for k, v in f.items()}
        e[name][at] += 0.5
        m = {k: v.clone() for k, v in f.items()}
        m[name][at] -= 0.5
        diff = (loss(e) - loss(m)).item()
        # grad_b takes the fp32 u it is given: off by u's own tolerance against the float64 u
        slack = 2 * D_LONG * STEP * 90 * 64 if name == "b" else 0.0
        assert abs(diff - got[name][at].item()) <= tol[at].item() + slack * 1e-2 + 1e-9, (name, at, diff, got[name][at])


def test_adapters_smaller_calls_and_no_tokens(e8q):
    """One object for calls of any size up to its limit; rows behind the last
    token are left as they were."""
    d = make(300, 136, 264, 16, 5)
    op = e8q.Lora(d["a"], d["b"], d["scale"], 300)
    for t in (300, 1, 128, 129, 64, 0):
        x, sl, base = d["x"][:t], d["slots"][:t], d["base"][:t]
        out = torch.full((t + 2, 264), 7.0, device="cuda", dtype=torch.bfloat16)
        u = torch.full((t + 2, 16), 7.0, device="cuda")
        op(x, sl, base=base, out=out[:t], u=u[:t])
        assert (out[t:] == 7).all() and (u[t:] == 7).all()
        sub = {k: (v[:t] if k in ("x", "slots", "base", "grad_y", "gx0") else v) for k, v in d.items()}
        if t:
            wy, ty, *_ = forward64(sub)
            close(out[:t], wy, ty, "y")
        outs = op.backward(d["grad_y"][:t], x, u[:t], sl, grad_x_base=d["gx0"][:t])
        for got, (want, tol), what in zip(outs, backward64(sub, u[:t]), ("grad_a", "grad_b", "grad_x")):
            close(got, want, tol, (t, what))


def test_adapters_on_other_streams_and_in_graphs(e8q):
    d = make(150, 264, 136, 16, 5)
    op = e8q.Lora(d["a"], d["b"], d["scale"], 150)
    y, u = (t.clone() for t in op(d["x"], d["slots"], base=d["base"], keep_u=True))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = e8q.Lora(d["a"], d["b"], d["scale"], 150)
    y2 = other(d["x"], d["slots"], base=d["base"], stream=side)
    side.synchronize()
    assert torch.equal(y, y2)
    graph = torch.cuda.CUDAGraph()
    out, uo = torch.empty_like(y), torch.empty_like(u)
    grads = [torch.empty_like(d["a"]), torch.empty_like(d["b"]), torch.empty_like(d["x"])]
    op.backward(d["grad_y"], d["x"], u, d["slots"])  # its workspace exists before the capture
    with torch.cuda.graph(graph):
        op(d["x"], d["slots"], base=d["base"], out=out, u=uo)
        op.backward(d["grad_y"], d["x"], uo, d["slots"], grad_x_base=d["gx0"], grad_a=grads[0], grad_b=grads[1],
                    grad_x=grads[2])
    fresh = e8q.Lora(d["a"], d["b"], d["scale"], 150)
    for seed in range(3):
        n = make(150, 264, 136, 16, 5, seed=seed + 1)
        for k in ("x", "slots", "base", "grad_y", "gx0", "a", "b", "scale"):
            d[k].copy_(n[k])
        graph.replay()
        torch.cuda.synchronize()
        y, u = fresh(d["x"], d["slots"], base=d["base"], keep_u=True)
        assert torch.equal(y, out) and torch.equal(u, uo)
        for a, b in zip(fresh.backward(d["grad_y"], d["x"], u, d["slots"], grad_x_base=d["gx0"]), grads):
            assert torch.equal(a, b)


@pytest.mark.parametrize("cols,rows", [(264, 136), (2304, 264)])
def test_adapters_replay_after_calls_of_other_sizes(e8q, cols, rows):
    """One captured call, then eager calls of every size on the same object:
    the captured one still has its workspace and its outputs."""
    T = 192
    d = make(T, cols, rows, 16, 5)
    op = e8q.Lora(d["a"], d["b"], d["scale"], T)
    fresh = e8q.Lora(d["a"], d["b"], d["scale"], T)
    op.backward(d["grad_y"][:1], d["x"][:1], op(d["x"][:1], d["slots"][:1], keep_u=True)[1], d["slots"][:1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, u = op(d["x"][:1], d["slots"][:1], base=d["base"][:1], keep_u=True)
        grads = op.backward(d["grad_y"][:1], d["x"][:1], u, d["slots"][:1])
    for t in (T, 130, 129, 128, 127, 100, 64, 40, 9, 2):
        sizes = (d["x"][:t], fresh(d["x"][:t], d["slots"][:t], keep_u=True)[1], d["slots"][:t])
        op(sizes[0], sizes[2], base=d["base"][:t], keep_u=True)
        op.backward(d["grad_y"][:t], *sizes)
        filler = torch.full((1 << 22,), float("nan"), device="cuda")  # takes any block that was given back
        graph.replay()
        torch.cuda.synchronize()
        wy, wu = fresh(d["x"][:1], d["slots"][:1], base=d["base"][:1], keep_u=True)
        assert torch.equal(y, wy) and torch.equal(u, wu) and bool(filler.isnan().all())
        for got, want in zip(grads, fresh.backward(d["grad_y"][:1], d["x"][:1], wu, d["slots"][:1])):
            assert torch.equal(got, want)


def test_adapters_past_32_bit_offsets(e8q):
    """The most tokens, and more than 2^31 elements in y and in x (4.3 GB each)."""
    T, wide = 65536, 32776
    for cols, rows in ((8, wide), (wide, 8)):
        g = torch.Generator("cuda").manual_seed(7)
        a, b = ((torch.randn(s, device="cuda", generator=g) * 0.1).bfloat16() for s in ((2, 8, cols), (2, rows, 8)))
        x = torch.ones((T, cols), device="cuda", dtype=torch.bfloat16)
        x[-3:] = 2
        slots = torch.zeros(T, dtype=torch.int32, device="cuda")
        slots[-2] = 1
        op = e8q.Lora(a, b, torch.ones(2, device="cuda"), T)
        y, u = op(x, slots, keep_u=True)
        gy = torch.zeros((T, rows), device="cuda", dtype=torch.bfloat16)
        gy[0], gy[-2:] = 1, 2
        ga, gb, gx = op.backward(gy, x, u, slots)
        for t in (0, T // 2, T - 3, T - 2, T - 1):
            i = int(slots[t])
            sub = dict(a=a[i:i + 1], b=b[i:i + 1], scale=torch.ones(1, device="cuda"), x=x[t:t + 1], grad_y=gy[t:t + 1],
                       base=torch.zeros((1, rows), device="cuda"), gx0=torch.zeros((1, cols), device="cuda"),
                       slots=torch.zeros(1, dtype=torch.int32, device="cuda"))
            wy, ty, wu, tu = forward64(sub, base=False)
            close(y[t:t + 1], wy, ty, "y")
            close(u[t:t + 1], wu, tu, "u")
            (w1, t1), (w2, t2), (wx, tx) = backward64(sub, u[t:t + 1])
            close(gx[t:t + 1], wx, tx, "grad_x")
            if i == 1:  # the only token of its adapter
                close(ga[1:], w1, t1, "grad_a")
                close(gb[1:], w2, t2, "grad_b")
        del x, y, gy, gx, op


def test_adapters_refuse_bad_tensors(e8q):
    d = make(10, 64, 72, 16, 3)
    for bad in (dict(a=d["a"].float()), dict(b=d["b"][:, :, :8].contiguous()), dict(scale=d["scale"].double()),
                dict(scale=d["scale"][:2]), dict(a=d["a"].cpu()), dict(a=d["a"][0]), dict(b=d["b"].transpose(1, 2)),
                dict(max_tokens=-1), dict(max_tokens=65537)):
        with pytest.raises(e8q.E8qError):
            e8q.Lora(**{**dict(a=d["a"], b=d["b"], scale=d["scale"], max_tokens=10), **bad})
    op = e8q.Lora(d["a"], d["b"], d["scale"], 10)
    odd = torch.zeros(10 * 64 + 1, device="cuda").bfloat16()[1:].view(10, 64)
    for bad in (dict(x=d["x"].float()), dict(x=d["x"][:9]), dict(slots=d["slots"].long()), dict(slots=d["slots"].view(2, 5)),
                dict(base=d["base"][:, :64].contiguous()), dict(base=d["base"].half()), dict(out=d["base"].float()),
                dict(u=torch.zeros((10, 8), device="cuda")), dict(x=odd), dict(x=d["x"].cpu()),
                dict(x=torch.cat([d["x"], d["x"]]), slots=torch.cat([d["slots"], d["slots"]]))):
        with pytest.raises(e8q.E8qError):
            op(**{**dict(x=d["x"], slots=d["slots"]), **bad})
    u = torch.zeros((10, 16), device="cuda")
    good = dict(grad_y=d["grad_y"], x=d["x"], u=u, slots=d["slots"])
    for bad in (dict(grad_y=d["grad_y"].float()), dict(u=u.bfloat16()), dict(u=u[:9]), dict(grad_x_base=d["base"]),
                dict(need_x=False, grad_x=torch.empty_like(d["x"])), dict(grad_x=d["x"]), dict(grad_a=d["a"]),
                dict(grad_b=torch.empty_like(d["b"]).float())):
        with pytest.raises(e8q.E8qError):
            op.backward(**{**good, **bad})
