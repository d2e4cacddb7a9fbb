"""Workloads of the row operators and the low-rank adapters: their inputs,
their plain forms in elementary torch operations, and the exact values.

Four operators around the 2-bit E8 matrices:

* ``lookup``       rows of an encoded matrix, chosen by token ids, decoded and
                   scaled (an embedding table held in the 2-bit form);
* ``lookup_grad``  the identity-STE gradient of that lookup: every latent row
                   gets the sum of the output gradients of its tokens;
* ``lora``         y[t] = base[t] + s_a B_a (A_a x_t), a = slots[t]: low-rank
                   adapters of many requests added to a shared projection;
* ``lora_grad``    the gradients of A, B and x.

``run`` computes the plain form where ``own`` is false and calls the library
where it is true.  Sizes: the widths of this repository's own workloads
(768, 2048, 4096, 14336) and generic token, row and adapter counts.
"""
from __future__ import annotations

import functools
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _lookup(name, n, rows, cols, block=0, basis="original", out="bf16", ids="i64", kappa=1.0, alpha=1.0, first=0):
    return dict(name=name, kind="lookup", n=n, rows=rows, cols=cols, block=block, basis=basis, out=out, ids=ids,
                kappa=kappa, alpha=alpha, first=first)


def _lgrad(name, n, rows, cols, grad="bf16", latent="bf16", ids="i64", alpha=1.0, first=0):
    return dict(name=name, kind="lookup_grad", n=n, rows=rows, cols=cols, grad=grad, latent=latent, ids=ids,
                alpha=alpha, first=first)


def _lora(name, kind, tokens, cols, rows, rank, adapters, ragged, train=False):
    return dict(name=name, kind=kind, tokens=tokens, cols=cols, rows=rows, rank=rank, adapters=adapters,
                ragged=ragged, train=train)


def listed():
    return [
        # one token of one request: the decode step of a single user
        _lookup("lookup, one token", 1, 32000, 4096, alpha=64.0),
        # a prefill chunk; weights quantised at kappa = 1 carry records in a fifth of their groups
        _lookup("lookup, prefill", 8192, 32000, 4096, alpha=64.0),
        # a shard of a wider table read in the rotated basis in fp32, odd sizes, half of the ids on other shards
        _lookup("lookup, shard in fp32", 4099, 25011, 768, basis="rotated", out="f32", ids="i32", kappa=0.6, first=12345),
        # a short fine-tuning batch into a mid-sized table
        _lgrad("lookup gradient, short batch", 96, 1000, 2048),
        # a training batch of natural-language tokens (a few rows hold most of them)
        _lgrad("lookup gradient, training", 16384, 32000, 4096, alpha=64.0),
        # an odd batch with fp32 gradients, into a shard of the table
        _lgrad("lookup gradient, shard in fp32", 5003, 25011, 768, grad="f32", latent="f32", ids="i32", first=12345),
        # one request decoding one token beside a 4096 x 4096 projection
        _lora("adapters, one token", "lora", 1, 4096, 4096, 16, 32, False),
        # a decode batch in which nearly every request has its own adapter, beside the MLP's wide projection
        _lora("adapters, decode batch", "lora", 64, 14336, 4096, 16, 64, False),
        # prompts of several requests in one batch; u is kept for the backward pass
        _lora("adapters, prefill", "lora", 4096, 4096, 14336, 32, 8, True, train=True),
        # three small adapters trained at once on an odd batch
        _lora("adapter gradients, small", "lora_grad", 257, 2048, 768, 8, 3, True),
        # a training step of four adapters
        _lora("adapter gradients, four", "lora_grad", 4096, 4096, 14336, 16, 4, True),
        # one adapter of a high rank on a long batch
        _lora("adapter gradients, one", "lora_grad", 8192, 14336, 4096, 64, 1, True),
    ]


WIDTHS = (64, 96, 256, 768, 1000, 2048, 4096, 5120, 14336)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("lookup", "lookup_grad", "lora", "lora_grad"))
    if kind in ("lookup", "lookup_grad"):
        cols = rng.choice(WIDTHS)
        n = min(_log(rng, 1, 16384), 8192 * 4096 // cols)
        rows = min(_log(rng, 200, 50000), 32000 * 4096 // cols)
        first = rng.choice((0, rng.randrange(1, 100000)))
        ids, alpha = rng.choice(("i32", "i64")), rng.choice((1.0, 0.5, math.sqrt(cols)))
        if kind == "lookup":
            c = _lookup("", n, rows, cols, basis=rng.choice(("original", "original", "rotated")),
                        block=rng.choice((0, 0, 0, 1, 8)), out=rng.choice(("bf16", "f32")), ids=ids,
                        kappa=rng.choice((0.6, 1.0)), alpha=alpha, first=first)
        else:
            c = _lgrad("", n, rows, cols, grad=rng.choice(("bf16", "f32")), latent=rng.choice(("bf16", "f32")), ids=ids,
                       alpha=alpha, first=first)
    else:
        cols, rows = rng.choice(WIDTHS), rng.choice(WIDTHS)
        adapters, rank = _log(rng, 1, 64), rng.choice((8, 16, 16, 24, 32, 64))
        adapters = min(adapters, 1024 // rank)
        tokens = min(_log(rng, 1, 8192), 4096 * 18432 // (cols + rows), 4096 * 256 // (adapters * rank))
        c = _lora("", kind, tokens, cols, rows, rank, adapters, rng.random() < 0.5, rng.random() < 0.5)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# the lattice (doubled coordinates P = 2p)
# --------------------------------------------------------------------------
def _key(P):
    """(|P|^2, then P lexicographically) as one integer; |P_i| <= 60."""
    w = torch.tensor([121 ** (7 - i) for i in range(8)], device=P.device, dtype=torch.int64)
    return P.square().sum(-1), ((P + 60) * w).sum(-1)


@functools.lru_cache(maxsize=1)
def _lattice():
    """The core (the first 65,536 points in norm, then lexicographic order)
    and the 240 roots, int64."""
    def grid(values):
        v = torch.tensor(values, device=DEV, dtype=torch.int64)
        half = torch.cartesian_prod(v, v, v, v)
        half = half[half.square().sum(1) <= 48]
        n2 = half.square().sum(1)
        i, j = torch.nonzero(n2[:, None] + n2[None, :] <= 48, as_tuple=True)
        P = torch.cat([half[i], half[j]], 1)
        return P[P.sum(1) % 4 == 0]

    P = torch.cat([grid(list(range(-6, 7, 2))), grid(list(range(-5, 6, 2)))])
    n2, lex = _key(P)
    P = P[torch.argsort(lex)]
    P = P[torch.argsort(P.square().sum(1), stable=True)]
    return P[:65536].contiguous(), P[1:241].contiguous()


def _rank(P):
    """Core index of each point, or -1."""
    core, _ = _lattice()
    n2, lex = _key(core)
    big = int(121 ** 8)
    out = torch.full(P.shape[:-1], -1, device=DEV, dtype=torch.int64)
    q2, qlex = _key(P)
    inside = q2 <= 48
    flat = torch.nonzero(inside.reshape(-1)).reshape(-1)
    q2f, qf = q2.reshape(-1)[flat], qlex.reshape(-1)[flat]
    comb = (n2 // 8) * big + lex          # |P|^2 is a multiple of 8: at most 6 * 121^8 < 2^63
    at = torch.searchsorted(comb, (q2f // 8) * big + qf).clamp(max=65535)
    hit = (n2[at] == q2f) & (lex[at] == qf)
    out.view(-1)[flat] = torch.where(hit, at, torch.full_like(at, -1))
    return out


def _nearest(x):
    """Nearest E8 point of x [n][8] (doubled), by rounding both cosets."""
    def d8(y):
        f = torch.round(y)
        d = y - f
        i = d.abs().argmax(1, keepdim=True)
        step = torch.where(d.gather(1, i) >= 0, 1.0, -1.0).to(y.dtype)
        odd = (f.sum(1, keepdim=True) % 2) != 0
        return f + torch.zeros_like(f).scatter(1, i, step) * odd

    a, b = d8(x), d8(x - 0.5) + 0.5
    nearer = ((x - b).square().sum(1) < (x - a).square().sum(1))[:, None]
    return torch.round(2 * torch.where(nearer, b, a)).to(torch.int64)


def _table(case, seed):
    """An encoded matrix and, apart from it, the points that it encodes."""
    g = torch.Generator(DEV).manual_seed(1000003 * seed + 17)
    rows, cols = case["rows"], case["cols"]
    gpr, pool = cols // 8, 32768
    x = torch.randn((pool, 8), device=DEV, generator=g, dtype=torch.float64) * case["kappa"]
    P = _nearest(x)
    core, roots = _lattice()
    idx = _rank(P)
    out = torch.nonzero(idx < 0).reshape(-1)
    root = torch.full((pool,), -1, device=DEV, dtype=torch.int64)
    if out.numel():
        r = _rank(P[out][:, None, :] - roots[None])
        r = torch.where(r < 0, torch.full_like(r, 1 << 20), r)
        best, which = r.min(1)
        found = best < (1 << 20)
        idx[out] = torch.where(found, best, torch.zeros_like(best))
        root[out] = torch.where(found, which, torch.full_like(which, -2))
    pick = torch.randint(0, pool, (rows, gpr), device=DEV, generator=g)
    r = root[pick]

    def records(mask):
        return torch.nonzero(mask.reshape(-1)).reshape(-1), torch.cat(
            [torch.zeros(1, device=DEV, dtype=torch.int64), mask.sum(1).cumsum(0)])

    def words(v):  # uint32 values in an int32 tensor
        return torch.where(v >= 1 << 31, v - (1 << 32), v).to(torch.int32)

    eg, erp = records(r >= 0)
    ep = pick.reshape(-1)[eg]
    esc = torch.stack([words(eg), words(idx[ep] | (root[ep] << 16))], 1)
    og, orp = records(r == -2)
    op = P[pick.reshape(-1)[og]].to(torch.int16).contiguous().view(torch.int32)
    ovf = torch.cat([words(og)[:, None], op.reshape(-1, 4)], 1)
    i16 = idx[pick]
    signs = torch.randint(0, 2, (cols,), device=DEV, generator=g) * 2 - 1
    scale = 0.02 / case["kappa"] * (0.8 + 0.4 * torch.rand(rows, device=DEV, generator=g))
    b = case["block"]
    if b == 0:
        b = min(cols & -cols, 2048)
    elif b > 1 and cols % b:
        b = 1
    m = dict(idx=torch.where(i16 >= 1 << 15, i16 - (1 << 16), i16).to(torch.int16), scale=scale.float(),
             signs=signs.to(torch.int8), esc=esc.contiguous().view(torch.uint8).reshape(-1), esc_row_ptr=erp,
             ovf=ovf.contiguous().view(torch.uint8).reshape(-1), ovf_row_ptr=orp, block=b)
    m["most"] = [int((p[1:] - p[:-1]).max()) for p in (erp, orp)]
    return m, P, pick


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
_T = {"bf16": torch.bfloat16, "f32": torch.float32, "i32": torch.int32, "i64": torch.int64}


def _ids(case, g):
    """Token ids with a natural-language-like skew (p ~ 1 / rank), every rank
    at a place of its own in the table; 1 % padding (-1), and for a shard
    as many ids again that live on other shards."""
    n, rows = case["n"], case["rows"]
    place = torch.randperm(rows, device=DEV, generator=g)
    rank = (torch.exp(torch.rand(n, device=DEV, generator=g) * math.log(rows + 1)) - 1).long().clamp(0, rows - 1)
    ids = place[rank] + case["first"]
    if case["first"]:
        away = torch.rand(n, device=DEV, generator=g) < 0.5
        ids = torch.where(away, torch.randint(0, case["first"], (n,), device=DEV, generator=g), ids)
    return torch.where(torch.rand(n, device=DEV, generator=g) < 0.01, torch.full_like(ids, -1), ids).to(_T[case["ids"]])


def _slots(case, g):
    """Adapter of every token: contiguous prompts of uneven lengths, or one
    token a request; about one in sixteen requests has no adapter (-1)."""
    t, a = case["tokens"], case["adapters"]
    req = torch.arange(t, device=DEV)
    if case["ragged"]:
        cuts = torch.rand(t, device=DEV, generator=g) < min(1.0, 2.0 * a / t)
        req = cuts.long().cumsum(0)
    which = torch.randint(0, a, (t + 1,), device=DEV, generator=g)
    which = torch.where(torch.rand(t + 1, device=DEV, generator=g) < 1 / 16, torch.full_like(which, -1), which)
    which[req[t // 2]] = 0
    return which[req].to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(DEV).manual_seed(seed)

    def rand(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(shape, device=DEV, generator=g) * std).to(dtype)

    s = dict(case=case)
    if case["kind"] == "lookup":
        m, _, _ = _table(case, seed)
        k = max(m["block"], 1).bit_length() - 1  # H_B as a product of two smaller ones
        s.update(m=m, ids=_ids(case, g), points=[v.float() for v in _lattice()],
                 h=[_hadamard(1 << q, torch.float32) for q in (k // 2, k - k // 2)])
        if own:
            from bit_e8_lattice_b200 import e8q

            s["encoded"] = e8q.Encoded(m["idx"], m["scale"], m["signs"], m["esc"], m["esc_row_ptr"], m["ovf"],
                                       m["ovf_row_ptr"], case["rows"], case["cols"], 0, m["block"],
                                       m["esc"].numel() // 8, m["ovf"].numel() // 20)
    elif case["kind"] == "lookup_grad":
        s.update(ids=_ids(case, g), grad=rand(case["n"], case["cols"], std=1e-3, dtype=_T[case["grad"]]))
        if own:
            from bit_e8_lattice_b200 import e8q

            s["op"] = e8q.RowsBackward(case["rows"], case["cols"], case["n"], grad_dtype=_T[case["grad"]],
                                       latent_dtype=_T[case["latent"]])
    else:
        t, k, n, r, a = (case[q] for q in ("tokens", "cols", "rows", "rank", "adapters"))
        s.update(x=rand(t, k), slots=_slots(case, g), a=rand(a, r, k, std=k ** -0.5), b=rand(a, n, r, std=r ** -0.5),
                 scale=0.5 + 1.5 * torch.rand(a, device=DEV, generator=g))
        if case["kind"] == "lora":
            s["base"] = rand(t, n)
        else:
            s.update(grad_y=rand(t, n, std=1e-2), grad_x_base=rand(t, k, std=1e-2))
            s["u"] = _down(s["x"], s["a"], s["slots"])
        if own:
            from bit_e8_lattice_b200 import e8q

            s["op"] = e8q.Lora(s["a"], s["b"], s["scale"], t)
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def _parity(v):
    v = v ^ (v >> 8)
    v = v ^ (v >> 4)
    v = v ^ (v >> 2)
    return (v ^ (v >> 1)) & 1


def _hadamard(n, dtype):
    i = torch.arange(n, device=DEV)
    return (1 - 2 * _parity(i[:, None] & i[None, :])).to(dtype)


def _row_records(rp, row, most):
    """Record numbers of the chosen rows, padded to `most` a row, and which of them are real."""
    start, count = rp[row], rp[row + 1] - rp[row]
    j = torch.arange(most, device=DEV)
    return start[:, None] + j, j < count[:, None]


def _plain_lookup(s):
    case, m = s["case"], s["m"]
    cols, rows, n = case["cols"], case["rows"], case["n"]
    gpr = cols // 8
    row = s["ids"].long() - case["first"]
    ok = (row >= 0) & (row < rows)
    row = torch.where(ok, row, torch.zeros_like(row))
    core, roots = s["points"]
    P = torch.zeros((n * gpr + 1, 8), device=DEV)
    P[:-1] = core[m["idx"][row].long() & 0xFFFF].reshape(-1, 8)
    at0 = torch.arange(n, device=DEV)[:, None] * gpr - row[:, None] * gpr
    if m["most"][0]:
        rec, real = _row_records(m["esc_row_ptr"], row, m["most"][0])
        w = m["esc"].view(torch.int32).view(-1, 2)[rec.clamp(max=m["esc"].numel() // 8 - 1)].long()
        at = torch.where(real, (w[..., 0] & 0xFFFFFFFF) + at0, n * gpr)
        P.index_add_(0, at.reshape(-1), roots[torch.where(real, (w[..., 1] >> 16) & 0xFF, 0)].reshape(-1, 8))
    if m["most"][1]:
        rec, real = _row_records(m["ovf_row_ptr"], row, m["most"][1])
        rec = rec.clamp(max=m["ovf"].numel() // 20 - 1)
        group = m["ovf"].view(torch.int32).view(-1, 5)[:, 0][rec].long() & 0xFFFFFFFF
        P[torch.where(real, group + at0, n * gpr).reshape(-1)] = \
            m["ovf"].view(torch.int16).view(-1, 10)[:, 2:][rec].reshape(-1, 8).float()
    P = P[:-1].reshape(n, cols)
    mul = m["scale"][row] * (0.5 * case["alpha"])
    if case["basis"] == "original":
        if m["block"] > 1:
            h1, h2 = s["h"]
            P = torch.matmul(torch.matmul(h1, P.reshape(-1, h1.shape[0], h2.shape[0])), h2).reshape(n, cols)
        mul = mul / math.sqrt(m["block"])
        P = P * m["signs"].float()
    return torch.where(ok[:, None], P * mul[:, None], torch.zeros_like(P)).to(_T[case["out"]])


def _plain_lookup_grad(s):
    case = s["case"]
    row = s["ids"].long() - case["first"]
    row = torch.where((row >= 0) & (row < case["rows"]), row, torch.full_like(row, case["rows"]))
    acc = torch.zeros((case["rows"] + 1, case["cols"]), device=DEV)
    acc.index_add_(0, row, s["grad"].float())
    return (acc[:-1] * case["alpha"]).to(_T[case["latent"]])


def _mask(slots, adapters):
    return (slots[:, None] == torch.arange(adapters, device=DEV)).float()


def _down(x, a, slots):
    """u[t] = A_a x_t: every adapter's product, of which each token keeps its own."""
    n, r, k = a.shape
    u = torch.matmul(x.float(), a.float().reshape(n * r, k).t()).reshape(-1, n, r)
    return (u * _mask(slots, n)[:, :, None]).sum(1)


def _spread(u, slots, adapters):
    """[t][adapters * r]: u in its own adapter's place, 0 in the others'."""
    return (u[:, None, :] * _mask(slots, adapters)[:, :, None]).reshape(u.shape[0], -1)


def _plain_lora(s):
    a, b, slots = s["a"], s["b"].float(), s["slots"]
    n, r = a.shape[0], a.shape[1]
    u = _down(s["x"], a, slots)
    scale = s["scale"][slots.clamp(min=0).long()]
    up = torch.matmul(_spread(u * scale[:, None], slots, n), b.transpose(1, 2).reshape(n * r, -1))
    y = (s["base"].float() + up).to(torch.bfloat16)
    return {"y": y, "u": u} if s["case"]["train"] else {"y": y}


def _plain_lora_grad(s):
    a, b, slots = s["a"].float(), s["b"].float(), s["slots"]
    n, r, k = a.shape
    scale = s["scale"][slots.clamp(min=0).long()][:, None]
    gy, x = s["grad_y"].float() * scale, s["x"].float()
    mask = _mask(slots, n)[:, :, None]
    v = torch.matmul(gy, b.transpose(0, 1).reshape(-1, n * r)).reshape(-1, n, r) * mask  # [t][adapter][r]
    v = v.reshape(-1, n * r)
    grad_a = torch.matmul(v.t(), x).reshape(n, r, k)
    grad_b = torch.matmul(gy.t(), _spread(s["u"], slots, n)).reshape(-1, n, r).transpose(0, 1)
    grad_x = s["grad_x_base"].float() + torch.matmul(v, a.reshape(n * r, k))
    return {"a": grad_a.to(torch.bfloat16), "b": grad_b.contiguous().to(torch.bfloat16), "x": grad_x.to(torch.bfloat16)}


def run(s):
    case = s["case"]
    kind = case["kind"]
    if not own:
        return {"lookup": _plain_lookup, "lookup_grad": _plain_lookup_grad, "lora": _plain_lora,
                "lora_grad": _plain_lora_grad}[kind](s)
    if kind == "lookup":
        from bit_e8_lattice_b200 import e8q

        return e8q.e8q_decode_rows(s["encoded"], s["ids"], case["basis"], alpha=case["alpha"], first_row=case["first"],
                                   out_dtype=_T[case["out"]])
    if kind == "lookup_grad":
        return s["op"](s["grad"], s["ids"], alpha=case["alpha"], first_row=case["first"])
    if kind == "lora":
        if case["train"]:
            y, u = s["op"](s["x"], s["slots"], base=s["base"], keep_u=True)
            return {"y": y, "u": u}
        return {"y": s["op"](s["x"], s["slots"], base=s["base"])}
    ga, gb, gx = s["op"].backward(s["grad_y"], s["x"], s["u"], s["slots"], grad_x_base=s["grad_x_base"])
    return {"a": ga, "b": gb, "x": gx}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    size = {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}
    if case["kind"] == "lookup":
        n, cols = case["n"], case["cols"]
        record = 0.197 * 8 + 0.019 * 20 if case["kappa"] == 1.0 else 0.01  # bytes of records a group
        b = case["block"] or min(cols & -cols, 2048)
        if b > 1 and cols % b:
            b = 1
        # a lookup's rows are read once each, however many tokens share one
        read = min(n, case["rows"]) * (cols // 8 * (2 + record) + 4 + 32)
        stages = math.log2(b) if case["basis"] == "original" else 0
        return {"bytes": read + n * (cols * size[case["out"]] + size[case["ids"]]), "flops": n * cols * (stages + 2)}
    if case["kind"] == "lookup_grad":
        n, cols = case["n"], case["cols"]
        return {"bytes": n * (cols * size[case["grad"]] + size[case["ids"]]) + case["rows"] * cols * size[case["latent"]],
                "flops": n * cols}
    t, k, n, r = (case[q] for q in ("tokens", "cols", "rows", "rank"))
    used = min(case["adapters"], t)
    weights = used * r * (k + n) * 2
    if case["kind"] == "lora":
        return {"bytes": t * (2 * k + 4 * n + 4) + weights + (4 * t * r if case["train"] else 0),
                "flops": 2 * t * r * (k + n)}
    return {"bytes": t * (2 * n + 6 * k + 4 * r + 4) + weights + case["adapters"] * r * (k + n) * 2,
            "flops": 4 * t * r * (k + n)}


# --------------------------------------------------------------------------
# exact values
# --------------------------------------------------------------------------
def _exact_lookup(case, seed):
    m, P, pick = _table(case, seed)
    ids = _ids(case, torch.Generator(DEV).manual_seed(seed)).long() - case["first"]
    ok = (ids >= 0) & (ids < case["rows"])
    y = torch.zeros((case["n"], case["cols"]), device=DEV, dtype=torch.float64)
    rows = ids[ok]
    p = (P[pick[rows]].double() / 2).reshape(rows.numel(), case["cols"]) * m["scale"][rows].double()[:, None]
    if case["basis"] == "original":
        b = m["block"]
        if b > 1:
            p = (p.reshape(-1, b) @ _hadamard(b, torch.float64)).reshape(p.shape) / math.sqrt(b)
        p = p * m["signs"].double()
    y[ok] = p * case["alpha"]
    return y


def _exact_lookup_grad(s):
    case = s["case"]
    y = torch.zeros((case["rows"], case["cols"]), device=DEV, dtype=torch.float64)
    order = torch.argsort(s["ids"].long(), stable=True)
    ids = s["ids"].long()[order] - case["first"]
    keep = (ids >= 0) & (ids < case["rows"])
    rows, count = torch.unique_consecutive(ids[keep], return_counts=True)
    g = s["grad"][order[keep]]
    for c in range(0, case["cols"], 512):  # in columns, so that the running sums fit
        sums = torch.cat([torch.zeros_like(g[:1, c:c + 512]).double(), g[:, c:c + 512].double().cumsum(0)])
        end = count.cumsum(0)
        y[rows, c:c + 512] = (sums[end] - sums[end - count]) * case["alpha"]
    return y


def _exact_lora(s):
    case = s["case"]
    train = s["case"]["train"]
    grad = case["kind"] == "lora_grad"
    out = {"y": s["base"].double()} if not grad else {"x": s["grad_x_base"].double()}
    if grad:
        out["a"], out["b"] = s["a"].double() * 0, s["b"].double() * 0
    elif train:
        out["u"] = torch.zeros((case["tokens"], case["rank"]), device=DEV, dtype=torch.float64)
    for a in range(case["adapters"]):
        t = torch.nonzero(s["slots"] == a).reshape(-1)
        if not t.numel():
            continue
        A, B, sc, x = s["a"][a].double(), s["b"][a].double(), s["scale"][a].double(), s["x"][t].double()
        if not grad:
            u = x @ A.t()
            out["y"][t] += sc * (u @ B.t())
            if train:
                out["u"][t] = u
        else:
            gy = s["grad_y"][t].double()
            v = sc * (gy @ B)
            out["a"][a] = v.t() @ x
            out["b"][a] = sc * (gy.t() @ s["u"][t].double())
            out["x"][t] += v @ A
    return out


def exact(case, seed):
    if case["kind"] == "lookup":
        return _exact_lookup(case, seed)
    s = prepare(case, seed)
    return _exact_lookup_grad(s) if case["kind"] == "lookup_grad" else _exact_lora(s)
