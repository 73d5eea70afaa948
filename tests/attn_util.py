"""Problems of paged attention for the tests: caches that hold NaN wherever no row may look."""

from __future__ import annotations

import numpy as np

from oracle import attn_oracle as ao

# One rounding to bf16: half a step, 2^-8 of the value. The weights of an output are rounded to bf16
# too: 2^-8 of the weighted magnitudes behind it. A score is D products summed in fp32, scaled by a
# rounded factor and its power of two taken: off by (D * 2^-24 + 2^-21) of the magnitudes in it, which
# moves a weight, and the sum of the weights, by that factor each. fp32 sums over up to 2^14 tokens, 16 or
# more of them at a time: 2^10 * 2^-24.
ROUND = 2.0 ** -8


def bound(out, spread, reach, D):
    score = (D * 2.0 ** -24 + 2.0 ** -21) * reach[..., None]
    return ROUND * np.abs(out) + (ROUND + 2 * score + 2.0 ** -13) * spread


def problem(torch, seed, lens, Hq, Hkv, D, page, order="nhd", holes=0.0, lead=0, tail=0, std=1.5):
    """lens: (new tokens, cached tokens) of each sequence; holes: share of pages given back; lead, tail:
    rows of q before the first sequence and behind the last. CPU tensors in a dict."""
    g = torch.Generator().manual_seed(seed)
    B = len(lens)
    width = max(1, max(-(-kv // page) for _, kv in lens)) + 1
    used = sum(-(-kv // page) for _, kv in lens)
    pages = used + 3
    ids = torch.randperm(pages, generator=g).tolist()
    table = torch.full((B, width), pages + 7, dtype=torch.int32)  # (past the cache: no page)
    shape = (pages, Hkv, page, D) if order == "hnd" else (pages, page, Hkv, D)
    k, v = (torch.full(shape, float("nan"), dtype=torch.bfloat16) for _ in range(2))
    kt, vt = (t.transpose(1, 2) if order == "hnd" else t for t in (k, v))
    at = 0
    for b, (n, kv) in enumerate(lens):
        for i in range(-(-kv // page)):
            if float(torch.rand(1, generator=g)) < holes:
                table[b, i] = -1 if i % 2 else pages
                continue
            p = ids[at]
            at += 1
            table[b, i] = p
            m = min(page, kv - i * page)
            kt[p, :m] = (torch.randn(m, Hkv, D, generator=g) * std).to(torch.bfloat16)
            vt[p, :m] = torch.randn(m, Hkv, D, generator=g).to(torch.bfloat16)
    starts = [lead]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    T = starts[-1] + tail
    q = (torch.randn(T, Hq, D, generator=g) * std).to(torch.bfloat16)
    plain = lead == 0 and tail == 0 and all(n == 1 for n, _ in lens)
    return dict(q=q, k=k, v=v, order=order, table=table, page=page,
                kv_lens=torch.tensor([kv for _, kv in lens], dtype=torch.int32),
                starts=None if plain else torch.tensor(starts, dtype=torch.int32))


def caches(p, device):
    k, v = p["k"].to(device), p["v"].to(device)
    return (k.transpose(1, 2), v.transpose(1, 2)) if p["order"] == "hnd" else (k, v)


def oracle(p, scale, window=0):
    k, v = caches(p, "cpu")
    f64 = lambda t: t.double().numpy()
    return ao.paged_attention(f64(p["q"]), f64(k), f64(v), p["table"].tolist(), p["kv_lens"].tolist(),
                              None if p["starts"] is None else p["starts"].tolist(), scale, window)


def check(got, want, spread, reach):
    """got: rows on the CPU. Rows of no sequence (NaN in want) are not looked at here."""
    got = got.double().numpy()
    of = ~np.isnan(want[:, 0, 0])
    err = np.abs(got[of] - want[of])
    bad = ~(err <= bound(want[of], spread[of], reach[of], want.shape[2]))
    assert not bad.any(), (f"rows {np.flatnonzero(of)[np.unique(np.argwhere(bad)[:, 0])][:8]}, "
                           f"{bad.sum()} values, worst {np.nanmax(np.where(bad, err, 0))}, "
                           f"not finite {int((~np.isfinite(got[of])).sum())}")
