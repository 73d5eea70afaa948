"""Cases of the attention half of a decoder layer: rotary positions, appending to a paged cache of
keys and values, and attention of the new tokens over it; each in a plain form and through the
library's entry points.

    rope     y = x with each pair (a, b) of its first R values turned by the token's angle:
             m * (a cos - b sin), m * (b cos + a sin), angle = position * inv_freq[i]
    append   cache_k[slot[t]] = rope(k[t]), cache_v[slot[t]] = v[t], and rope(q[t]) beside them
    attend   out[r, h] = sum_j softmax_j(scale * q[r, h] . k[j]) v[j]
             over the cached tokens j that row r sees

Pairs are (i, i + R/2) in the half layout and (2i, 2i + 1) in the interleaved one. The cache is
[page, token of the page, head, D], or [page, head, token of the page, D] in memory (order "hnd");
a sequence's tokens lie on the pages that its row of the page table names. The chunk's tokens are a
sequence's last ones: row i of q of them sits at position kv - q + i and sees the positions up to its
own (the last `window` of them where window > 0) that lie on a page; a row that sees none is 0.

`own` false: elementary torch operations in 32 bits (angles in 64). `own` true: the library's calls.
"""

import math
import random

import torch

own = False


# ------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # queries of a decoding step of 23 requests, whole heads: one small launch
        dict(name="rope-decode", op="rope", T=23, heads=16, D=128, R=128, inter=False, far=4096,
             scaled=False, strided=False),
        # a prefill chunk at far positions of a context scaled beyond the trained one, half of each
        # head, queries inside the rows of a joint projection
        dict(name="rope-prefill", op="rope", T=8192, heads=32, D=128, R=64, inter=True, far=1 << 20,
             scaled=True, strided=True),
        # the decoding step's keys and values into pages of 16, its queries on the way
        dict(name="append-decode", op="append", T=23, Hq=16, Hkv=2, D=128, R=128, inter=False,
             far=4096, scaled=False, page=16, order="nhd", pad=0.0, q=True),
        # a padded prefill chunk into pages of 64, the rows one joint projection
        dict(name="append-prefill", op="append", T=8192, Hq=32, Hkv=4, D=128, R=64, inter=True,
             far=1 << 20, scaled=True, page=64, order="hnd", pad=0.1, q=True),
        # one request alone
        dict(name="attend-one-token", op="attend", B=1, q=1, kv=2000, Hq=16, Hkv=2, D=128, page=16,
             order="nhd", window=0, ragged="none"),
        # a decoding step: 23 requests of unlike lengths, captured for 24
        dict(name="attend-decode", op="attend", B=24, q=1, kv=8191, Hq=16, Hkv=2, D=128, page=16,
             order="nhd", window=0, ragged="decode"),
        # a few requests with very long contexts
        dict(name="attend-decode-long", op="attend", B=4, q=1, kv=131072, Hq=64, Hkv=8, D=128,
             page=64, order="hnd", window=0, ragged="none"),
        # sixteen requests with six verify tokens each, four query heads a key head
        dict(name="attend-verify", op="attend", B=16, q=6, kv=6000, Hq=32, Hkv=8, D=64, page=32,
             order="nhd", window=0, ragged="chunks"),
        # a chunk of a long prompt over what is cached already: few rows, a long axis
        dict(name="attend-chunk", op="attend", B=1, q=509, kv=30001, Hq=32, Hkv=4, D=128, page=16,
             order="nhd", window=0, ragged="none"),
        # prompts, chunks and decoding requests in one batch, a sliding window, pages before it gone
        dict(name="attend-mixed-window", op="attend", B=19, q=1500, kv=9000, Hq=32, Hkv=8, D=64,
             page=64, order="hnd", window=1024, ragged="mixed"),
        # a whole prompt
        dict(name="attend-prompt", op="attend", B=1, q=8192, kv=8192, Hq=32, Hkv=4, D=128, page=64,
             order="nhd", window=0, ragged="none"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend", "attend"])
    while True:
        D = rng.choice([64, 64, 128, 128, 128, 256])
        turn = dict(R=rng.choice([D, D, D // 2, D // 4]), inter=rng.random() < 0.5,
                    far=_log(rng, 64, 1 << 20), scaled=rng.random() < 0.4)
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 7, 8, 8, 16])
        page, order = rng.choice([1, 8, 16, 16, 32, 64, 64, 128]), rng.choice(["nhd", "hnd"])
        if op == "rope":
            c = dict(op=op, T=_log(rng, 1, 8192), heads=Hq, D=D, strided=rng.random() < 0.5, **turn)
            if c["T"] * Hq * D <= 8192 * 32 * 128:
                return c
        elif op == "append":
            c = dict(op=op, T=_log(rng, 1, 8192), Hq=Hq, Hkv=Hkv, D=D, page=page, order=order,
                     pad=rng.choice([0.0, 0.1]), q=rng.random() < 0.7, **turn)
            if c["T"] * (Hq + 2 * Hkv) * D <= 8192 * 40 * 128:
                return c
        else:
            kind = rng.choice(["decode", "decode", "chunks", "chunks", "mixed", "none"])
            B = _log(rng, 1, 200) if kind != "none" else rng.randint(1, 4)
            kv = _log(rng, 1, 131072)
            q = 1 if kind == "decode" else min(kv, _log(rng, 2, 16) if kind == "chunks" else
                                               _log(rng, 1, 8192))
            c = dict(op=op, B=B, q=q, kv=kv, Hq=Hq, Hkv=Hkv, D=D, page=page, order=order,
                     window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]), ragged=kind)
            need = work(c)
            if (need["flops"] <= 5.5e11 and Hkv * D * sum(k for _, k in _lengths(c)) <= 1 << 29
                    and sum(n for n, _ in _lengths(c)) <= 16384):
                return c


def _lengths(c):
    """(new tokens, cached tokens) of each sequence; a case has them, whatever the seed."""
    rng = random.Random(c["B"] * 1000003 + c["kv"] * 101 + c["q"])
    out = [(c["q"], c["kv"])]
    for i in range(1, c["B"]):
        if c["ragged"] == "none":
            out.append((c["q"], c["kv"]))
            continue
        kv = _log(rng, max(1, c["kv"] // 16), c["kv"])
        if c["ragged"] == "mixed":
            out.append((rng.choice([1, 1, 1, min(kv, _log(rng, 1, c["q"]))]), kv))
        else:
            out.append((min(kv, rng.randint(1, c["q"])), kv))
    if c["ragged"] in ("decode", "mixed") and c["B"] > 2:
        out[-1] = (1, 0)  # a row that only fills the batch up
    return out


# -------------------------------------------------------------------------------------- the inputs
def _inv_freq(c):
    """fp32 [R / 2]: base 10000; scaled: the slow half of the frequencies divided by 8, the fast
    quarter kept, a ramp between them, as contexts are stretched by parts."""
    n = c["R"] // 2
    f = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    if c["scaled"]:
        keep = (2.0 - 4.0 * torch.arange(n, dtype=torch.float64) / n).clamp(0.0, 1.0)
        f = f * (keep + (1.0 - keep) / 8.0)
    return f.to(torch.float32).cuda()


def _normal(g, shape, std=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        n = min(1 << 28, flat.numel() - i)
        flat[i:i + n] = torch.randn(n, generator=g, device="cuda").mul_(std)
    return out


def _cache(c, g, pages, std=1.0):
    """[pages, page, Hkv, D], filled with what other sequences left there."""
    if c["order"] == "hnd":
        return _normal(g, (pages, c["Hkv"], c["page"], c["D"]), std).transpose(1, 2)
    return _normal(g, (pages, c["page"], c["Hkv"], c["D"]), std)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    D = c["D"]
    if c["op"] != "attend":
        T = c["T"]
        s = dict(c=c, inv_freq=_inv_freq(c), m=1.0 + 0.1 * math.log(8.0) if c["scaled"] else 1.0)
        s["positions"] = torch.randint(c["far"], (T,), generator=g, device="cuda").to(torch.int32)
    if c["op"] == "rope":
        wide = c["heads"] + 8 if c["strided"] else c["heads"]
        s["x"] = _normal(g, (T, wide, D), 2.0)[:, :c["heads"]]
        return s
    if c["op"] == "append":
        Hq, Hkv = c["Hq"] if c["q"] else 0, c["Hkv"]
        rows = _normal(g, (T, Hq + 2 * Hkv, D), 2.0)  # one joint projection
        s["q"] = rows[:, :Hq] if c["q"] else None
        s["k"], s["v"] = rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
        pages = -(-T // c["page"]) + 3
        slots = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        slots = slots.unsqueeze(1) * c["page"] + torch.arange(c["page"], device="cuda",
                                                              dtype=torch.int32)
        slots = slots.view(-1)[:T].clone()
        if c["pad"]:
            slots[T - int(T * c["pad"]):] = -1  # rows behind the last token
        s["slots"] = slots
        s["k_cache"], s["v_cache"] = _cache(c, g, pages), _cache(c, g, pages)
        return s
    lens = _lengths(c)
    T = sum(n for n, _ in lens)
    s = dict(c=c, lens=lens, scale=D ** -0.5, window=c["window"])
    # queries and keys of like direction now and then: a softmax that is not flat
    s["q"] = _normal(g, (T, c["Hq"], D), 1.5)
    width = max(1, max(-(-kv // c["page"]) for _, kv in lens))
    total = sum(-(-kv // c["page"]) for _, kv in lens)
    order = torch.randperm(total + 5, generator=g, device="cuda").to(torch.int32).tolist()
    table, at = [], 0
    for n, kv in lens:
        here = -(-kv // c["page"])
        row = order[at:at + here] + [-1] * (width - here)
        at += here
        if c["window"]:  # pages that no row sees any more have been given back
            gone = max(0, kv - n - c["window"] + 1) // c["page"]
            row[:gone] = [-1] * gone
        table.append(row)
    s["table"] = torch.tensor(table, dtype=torch.int32, device="cuda")
    s["k_cache"], s["v_cache"] = _cache(c, g, total + 5, 1.5), _cache(c, g, total + 5)
    s["kv_lens"] = torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda")
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    s["starts"] = None
    if any(n != 1 for n, _ in lens):
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------------ one pass
def run(state):
    return _library(state) if own else _plain(state)


def _library(s):
    import moe_lora_virtual_gb300 as mol

    op = s["c"]["op"]
    if op == "attend":
        return mol.mol_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"],
                                       s["starts"], scale=s["scale"], window=s["window"])
    rope = mol.Rope(s["inv_freq"], s["c"]["inter"], s["m"])
    if op == "rope":
        return mol.mol_rope(s["x"], s["positions"], rope)
    q = mol.mol_cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"],
                             positions=s["positions"], rope=rope, q=s["q"])
    return (s["k_cache"], s["v_cache"]) + (() if q is None else (q,))


def _turn(x, s):
    """fp32 rows [T, heads, D] with their positions turned into them."""
    x, R = x.to(torch.float32), s["c"]["R"]
    angle = s["positions"].to(torch.float64).unsqueeze(1) * s["inv_freq"].to(torch.float64)
    cos = (angle.cos() * s["m"]).to(torch.float32).unsqueeze(1)
    sin = (angle.sin() * s["m"]).to(torch.float32).unsqueeze(1)
    out = x.clone()
    if s["c"]["inter"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        out[..., 0:R:2], out[..., 1:R:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        out[..., :R // 2], out[..., R // 2:R] = a * cos - b * sin, b * cos + a * sin
    return out


def _plain(s):
    c = s["c"]
    if c["op"] == "rope":
        return _turn(s["x"], s).to(torch.bfloat16)
    if c["op"] == "append":
        keep = s["slots"] >= 0
        at = s["slots"][keep].to(torch.int64)
        page, token = at // c["page"], at % c["page"]
        s["k_cache"][page, token] = _turn(s["k"], s)[keep].to(torch.bfloat16)
        s["v_cache"][page, token] = s["v"][keep]
        out = (s["k_cache"], s["v_cache"])
        return out + ((_turn(s["q"], s).to(torch.bfloat16),) if c["q"] else ())
    Hkv, D, group = c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    out = torch.zeros_like(s["q"])
    at = 0
    for b, (n, kv) in enumerate(s["lens"]):
        first = 0
        if s["window"]:
            first = max(0, kv - n - s["window"] + 1) // c["page"]
        pages = s["table"][b, first:-(-kv // c["page"])].to(torch.int64)
        first *= c["page"]
        k, v = (t[pages.clamp(min=0)].reshape(-1, Hkv, D)[:kv - first].to(torch.float32)
                .transpose(0, 1) for t in (s["k_cache"], s["v_cache"]))
        held = (pages >= 0).repeat_interleave(c["page"])[:kv - first]
        j = torch.arange(first, kv, device=held.device)
        step = max(1, (1 << 27) // max(1, c["Hq"] * (kv - first)))
        for r in range(0, n if kv > first else 0, step):
            m = min(step, n - r)
            q = s["q"][at + r:at + r + m].to(torch.float32).view(m, Hkv, group, D)
            q = q.permute(1, 0, 2, 3).reshape(Hkv, m * group, D)
            own_at = torch.arange(kv - n + r, kv - n + r + m, device=j.device).unsqueeze(1)
            sees = (j <= own_at) & held
            if s["window"]:
                sees &= j > own_at - s["window"]
            sees = sees.repeat_interleave(group, 0)
            x = torch.bmm(q, k.transpose(1, 2)).mul_(s["scale"])
            x.masked_fill_(~sees, -math.inf)
            top = x.amax(2, keepdim=True).clamp_(min=-3.0e38)
            p = x.sub_(top).exp_()
            total = p.sum(2, keepdim=True)
            o = torch.bmm(p, v) / torch.where(total == 0, 1.0, total)
            o = o.view(Hkv, m, group, D).permute(1, 0, 2, 3)
            out[at + r:at + r + m] = o.reshape(m, c["Hq"], D).to(torch.bfloat16)
        at += n
    return out


# ---------------------------------------------------------------------------------- what it takes
def work(case):
    c = case
    if c["op"] == "rope":
        return dict(bytes=c["T"] * (4.0 * c["heads"] * c["D"] + 4) + 2.0 * c["R"],
                    flops=3.0 * c["T"] * c["heads"] * c["R"])
    if c["op"] == "append":
        T = c["T"] - int(c["T"] * c["pad"])
        Hq = c["Hq"] if c["q"] else 0
        return dict(bytes=4.0 * c["D"] * (c["T"] * Hq + 2 * T * c["Hkv"]) + 8.0 * T + 2.0 * c["R"],
                    flops=3.0 * c["R"] * (c["T"] * Hq + T * c["Hkv"]))
    pairs = tokens = rows = 0
    for n, kv in _lengths(c):
        w, first = c["window"] or kv, kv - n + 1       # the first row sees `first` positions
        full = max(0, min(n, kv - max(w, first) + 1))  # rows that see w of them
        part = n - full
        pairs += full * w + part * max(0, first + first + part - 1) // 2 if kv else 0
        tokens += min(kv, w + n - 1)
        rows += n
    return dict(bytes=4.0 * c["D"] * (rows * c["Hq"] + tokens * c["Hkv"]),
                flops=4.0 * c["Hq"] * c["D"] * pairs)


# --------------------------------------------------------------------------------------- 64 bits
def _turn64(x, s):
    x, R = x.double(), s["c"]["R"]
    n = R // 2
    first = torch.arange(n, device=x.device)
    first, second = (2 * first, 2 * first + 1) if s["c"]["inter"] else (first, first + n)
    angle = torch.outer(s["positions"].double(), s["inv_freq"].double())[:, None]
    turned = torch.view_as_complex(torch.stack([x[..., first], x[..., second]], -1))
    turned = turned * torch.polar(torch.full_like(angle, s["m"]), angle)
    out = x.clone()
    out[..., first], out[..., second] = turned.real, turned.imag
    return out


def exact(case, seed):
    c = case
    if c["op"] == "attend":  # every row against every token of its sequence that has a page
        pairs = sum(n * min(kv, (c["window"] or kv) + n + c["page"]) for n, kv in _lengths(c))
        if 4.0 * pairs * c["Hq"] * c["D"] > 2e12:
            return None
    s = prepare(case, seed)
    if c["op"] == "rope":
        return _turn64(s["x"], s)
    if c["op"] == "append":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        turned, given = _turn64(s["k"], s), s["v"].double()
        rows = torch.nonzero(s["slots"] >= 0).view(-1)
        at = s["slots"][rows].long()
        where = (torch.div(at, c["page"], rounding_mode="floor"), at.remainder(c["page"]))
        k.index_put_(where, turned[rows])
        v.index_put_(where, given[rows])
        return (k, v) + ((_turn64(s["q"], s),) if c["q"] else ())
    group, at = c["Hq"] // c["Hkv"], 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    pages = s["table"].tolist()
    for b, (n, kv) in enumerate(s["lens"]):
        tokens = [j for j in range(kv) if pages[b][j // c["page"]] >= 0]
        rows, at = slice(at, at + n), at + n
        if not tokens:
            continue
        where = torch.tensor([pages[b][j // c["page"]] for j in tokens], device="cuda")
        tokens = torch.tensor(tokens, device="cuda")
        offset = tokens % c["page"]
        place = torch.arange(kv - n, kv, device="cuda")
        for h in range(c["Hkv"]):
            k, v = s["k_cache"][where, offset, h].double(), s["v_cache"][where, offset, h].double()
            for i in range(h * group, (h + 1) * group):
                q = s["q"][rows, i].double()
                for r in range(0, n, 1024):
                    p = place[r:r + 1024, None]
                    hidden = tokens[None] > p
                    if s["window"]:
                        hidden |= tokens[None] <= p - s["window"]
                    x = (q[r:r + 1024] @ k.T * s["scale"]).masked_fill(hidden, -math.inf)
                    w = torch.nan_to_num(torch.softmax(x, 1), nan=0.0)
                    out[rows, i][r:r + 1024] = w @ v
    return out
