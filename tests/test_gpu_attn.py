"""GPU tests of the attention half of a layer against the float64 oracle.

Rotation: one rounding to bf16, 2^-8 of the value, and sines off by 2^-21 with products in fp32,
2^-19 of the pair's magnitudes. The bounds of attention: tests/attn_util.py.
"""

import numpy as np
import pytest

from oracle import attn_oracle as ao
from tests import attn_util as au
from tests.gpu_util import mol_lib, torch_cuda

pytestmark = pytest.mark.gpu

ROUND = 2.0 ** -8


@pytest.fixture(scope="module")
def env():
    return torch_cuda(), mol_lib()


def f64(t):
    return t.detach().double().cpu().numpy()


def turned(torch, x, positions, rope):
    """(exact rows, their bound)"""
    n = rope.inv_freq.shape[0]
    want = ao.rope(f64(x), f64(positions), f64(rope.inv_freq), rope.interleaved, rope.magnitude)
    mag = np.abs(f64(x))[..., :2 * n]
    pair = mag.copy()
    if rope.interleaved:
        pair[..., ::2] = pair[..., 1::2] = mag[..., ::2] + mag[..., 1::2]
    else:
        pair[..., :n] = pair[..., n:] = mag[..., :n] + mag[..., n:]
    bound = np.zeros_like(want)
    bound[..., :2 * n] = ROUND * np.abs(want[..., :2 * n]) + 2.0 ** -19 * pair * abs(rope.magnitude)
    return want, bound


def near(got, want, bound):
    err = np.abs(f64(got) - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{np.argwhere(bad)[:4].tolist()} off by {err[bad][:4]}"


def randn(torch, g, *shape):
    return (torch.randn(*shape, generator=g) * 2).to(torch.bfloat16)


# -------------------------------------------------------------------------------------- positions
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,H,D,R,layout", [
    (1, 1, 16, 16, "plain"), (23, 16, 128, 128, "plain"), (5, 3, 128, 32, "strided"),
    (130, 7, 80, 48, "in place"), (4, 40, 256, 64, "heads first"), (9, 2, 512, 512, "strided"),
    (7, 5, 72, 16, "plain")])
def test_rope(env, T, H, D, R, layout, interleaved):
    torch, mol = env
    g = torch.Generator().manual_seed(T * H + R)
    rope = mol.rope_frequencies(R, interleaved=interleaved, magnitude=1.25, device="cuda")
    x = randn(torch, g, T, H, D)
    positions = torch.randint(-(1 << 31), (1 << 31) - 1, (T,), generator=g).to(torch.int32)
    positions[0] = 0
    positions[T // 2:] = torch.randint(1 << 20, (T - T // 2,), generator=g).to(torch.int32)
    dx, out = x.cuda(), None
    if layout == "strided":
        wide = torch.full((T, H + 2, D + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[:, :H, :D] = dx
        dx = wide[:, :H, :D]
        out = torch.full((T, H + 1, D + 16), 7.0, dtype=torch.bfloat16, device="cuda")[:, :H, :D]
    elif layout == "heads first":
        dx = dx.transpose(0, 1).contiguous().transpose(0, 1)
    elif layout == "in place":
        out = dx
    got = mol.mol_rope(dx, positions.cuda(), rope, out=out)
    near(got, *turned(torch, x, positions, rope))
    if layout == "strided":
        wide = got.as_strided((T, H + 1, D + 16), (got.stride(0), got.stride(1), 1))
        assert bool((wide[:, H:] == 7).all()) and bool((wide[..., D:] == 7).all())


# ------------------------------------------------------------------------------------------ append
@pytest.mark.parametrize("order", ["nhd", "hnd", "joint"])
@pytest.mark.parametrize("T,Hq,Hkv,D,R,page,interleaved", [
    (1, 1, 1, 64, 64, 1, False), (23, 16, 2, 128, 128, 16, False), (77, 10, 5, 64, 32, 7, True),
    (300, 0, 3, 256, 64, 64, True), (12, 4, 2, 128, 0, 16, False)])
def test_append(env, T, Hq, Hkv, D, R, page, interleaved, order):
    torch, mol = env
    g = torch.Generator().manual_seed(T + D)
    pages = -(-T // page) + 2
    if order == "joint":  # keys and values of a page in one buffer
        both = torch.full((pages, 2, page, Hkv, D), 3.0, dtype=torch.bfloat16, device="cuda")
        kc, vc = both[:, 0], both[:, 1]
    else:
        shape = (pages, Hkv, page, D) if order == "hnd" else (pages, page, Hkv, D)
        kc, vc = (torch.full(shape, 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        if order == "hnd":
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    rows = randn(torch, g, T, Hq + 2 * Hkv, D)
    k, v = rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    if T > 4:
        slots[1], slots[2], slots[3] = -1, pages * page, (1 << 31) - 1
    positions = torch.randint(1 << 20, (T,), generator=g).to(torch.int32)
    rope = mol.rope_frequencies(R, interleaved=interleaved, device="cuda") if R else None
    drows = rows.cuda()
    q = drows[:, :Hq] if Hq and R else None
    got = mol.mol_cache_append(drows[:, Hq:Hq + Hkv], drows[:, Hq + Hkv:], kc, vc, slots.cuda(),
                               positions.cuda() if R else None, rope, q=q)
    tk, bk = turned(torch, k, positions, rope) if R else (f64(k), np.zeros(k.shape))
    before = np.full(kc.shape, 3.0)
    wk, wv = ao.cache_append(tk, f64(v), before, before, slots.tolist())
    near(kc, wk, ao.cache_append(bk, f64(v), 0 * before, before, slots.tolist())[0])
    assert np.array_equal(f64(vc), wv)
    if q is None:
        assert got is None
    else:
        near(got, *turned(torch, rows[:, :Hq], positions, rope))


def test_append_turns_queries_in_place(env):
    torch, mol = env
    g = torch.Generator().manual_seed(5)
    rows, positions = randn(torch, g, 9, 8, 64), torch.arange(9, dtype=torch.int32) * 1000
    rope = mol.rope_frequencies(64, device="cuda")
    kc, vc = (torch.zeros(3, 4, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    d = rows.cuda()
    q = d[:, :4]
    got = mol.mol_cache_append(d[:, 4:6], d[:, 6:], kc, vc, torch.arange(9, dtype=torch.int32).cuda(),
                               positions.cuda(), rope, q=q, q_out=q)
    assert got is q
    near(d[:, :4], *turned(torch, rows[:, :4], positions, rope))
    assert torch.equal(d[:, 4:].cpu(), rows[:, 4:])


# --------------------------------------------------------------------------------------- attention
def attend(env, p, window=0, scale=None, fill=9.0, **kw):
    torch, mol = env
    D = p["q"].shape[2]
    kc, vc = au.caches(p, "cuda")
    out = torch.full(p["q"].shape, fill, dtype=torch.bfloat16, device="cuda")
    got = mol.mol_paged_attention(p["q"].cuda(), kc, vc, p["table"].cuda(), p["kv_lens"].cuda(),
                                  None if p["starts"] is None else p["starts"].cuda(),
                                  scale=scale, window=window, out=out, **kw)
    assert got is out
    return got.cpu()


def run(env, p, window=0, scale=None, fill=9.0):
    D = p["q"].shape[2]
    want, spread, reach = au.oracle(p, D ** -0.5 if scale is None else scale, window)
    got = attend(env, p, window, scale, fill)
    au.check(got, want, spread, reach)
    rest = np.isnan(want[:, 0, 0])
    assert bool((got[rest] == fill).all())  # rows of no sequence stay as they were
    return got


SHAPES = [  # Hq, Hkv, D, page, order
    (16, 2, 128, 16, "nhd"), (4, 4, 64, 64, "hnd"), (5, 1, 128, 1, "nhd"), (14, 2, 64, 8, "hnd"),
    (8, 1, 256, 16, "nhd"), (64, 2, 128, 32, "hnd"), (12, 3, 64, 5, "nhd"), (64, 1, 64, 128, "nhd"),
    (6, 3, 256, 128, "hnd")]


@pytest.mark.parametrize("Hq,Hkv,D,page,order", SHAPES)
@pytest.mark.parametrize("lens", [[1], [2, 0, 17], [64, 63, 65, 1, 128, 129, 0, 500], [3001, 5]])
def test_one_token_each(env, Hq, Hkv, D, page, order, lens):
    torch, _ = env
    run(env, au.problem(torch, sum(lens) + D, [(1, n) for n in lens], Hq, Hkv, D, page, order))


@pytest.mark.parametrize("Hq,Hkv,D,page,order", SHAPES)
@pytest.mark.parametrize("window", [0, 1, 70])
def test_chunks(env, Hq, Hkv, D, page, order, window):
    """Verify chunks, a prompt of its own, more rows than cached tokens, empty sequences."""
    torch, _ = env
    lens = [(3, 200), (1, 77), (0, 40), (40, 40), (6, 4), (2, 0), (17, 300), (0, 0), (1, 1)]
    run(env, au.problem(torch, Hq * D + window, lens, Hq, Hkv, D, page, order), window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 24])
@pytest.mark.parametrize("lens", [[(150, 150)], [(200, 520), (1, 300), (131, 131)], [(129, 1100)]])
def test_prompts(env, D, page, lens):
    torch, _ = env
    run(env, au.problem(torch, D + page, lens, 4, 2, D, page), 0)
    run(env, au.problem(torch, D + page, lens, 8, 1, D, page, "hnd", lead=3, tail=5), 100)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 16, 2), (256, 4, 2)])
def test_pages_given_back(env, D, Hq, Hkv):
    """Holes anywhere: tokens that no row sees; rows whose every page is gone are 0."""
    torch, _ = env
    lens = [(1, 100), (1, 900), (5, 333), (70, 400), (1, 3), (8, 16), (200, 200)]
    run(env, au.problem(torch, D, lens, Hq, Hkv, D, 16, holes=0.5))
    p = au.problem(torch, D, lens, Hq, Hkv, D, 16, holes=1.1)
    assert bool((run(env, p) == 0).all())


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 2), (128, 16, 2), (128, 3, 3), (256, 4, 2)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("window", [0, 40])
def test_what_a_row_does_not_see_does_not_reach_it(env, D, Hq, Hkv, bad, window):
    """A value that is not finite among a chunk's own tokens: rows before it, and past the window, are
    as if it were not there; those that see it are not finite."""
    torch, _ = env
    for lens in ([(6, 70), (1, 33)], [(180, 300), (1, 5)]):
        p = au.problem(torch, D + 1, lens, Hq, Hkv, D, 16)
        clean, spread, reach = au.oracle(p, D ** -0.5, window)
        n, kv = lens[0]
        at = kv - n // 2  # position of a token in the middle of the chunk
        page, offset = int(p["table"][0, at // 16]), at % 16
        for which in ("k", "v"):
            hurt = dict(p, **{which: p[which].clone()})
            hurt[which][page, offset, :, 3] = bad
            got = attend(env, hurt, window)
            i = np.arange(n)
            sees = (kv - n + i >= at) & ((window == 0) | (kv - n + i - window < at))
            others = np.ones(p["q"].shape[0], bool)
            others[:n] = ~sees
            want = np.where(others[:, None, None], clean, np.nan)
            au.check(got, want, spread, reach)
            if which == "v" and bad != bad:
                assert bool(torch.isnan(got[:n][torch.from_numpy(sees)][..., 3]).all())
            if which == "v":
                assert not bool(torch.isfinite(got[:n][torch.from_numpy(sees)][..., 3]).any())


def test_table_and_lengths_past_their_ends(env):
    """Lengths past the table are its width; starts past the rows are their end; none below 0."""
    torch, mol = env
    p = au.problem(torch, 3, [(1, 64), (2, 48)], 4, 2, 64, 16)
    p["table"] = p["table"][:, :4].contiguous()
    want = au.oracle(p, 0.125)
    long = dict(p, kv_lens=torch.tensor([1 << 30, 48], dtype=torch.int32))
    au.check(attend(env, long), *want)
    long = dict(p, starts=torch.tensor([-4, 1, 1 << 30], dtype=torch.int32))
    au.check(attend(env, long), *want)
    none = dict(p, kv_lens=torch.tensor([-5, -(1 << 31)], dtype=torch.int32))
    assert bool((attend(env, none) == 0).all())


def test_no_rows_no_sequences_no_pages(env):
    torch, mol = env
    bf = dict(dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    kc = torch.zeros(2, 16, 2, 64, **bf)
    table = torch.zeros(1, 1, **i32)
    lens = torch.ones(1, **i32)
    assert mol.mol_paged_attention(torch.zeros(0, 4, 64, **bf), kc, kc, table[:0], lens[:0]).shape == (0, 4, 64)
    out = torch.full((3, 4, 64), 5.0, **bf)
    mol.mol_paged_attention(out, kc, kc, table, lens, torch.zeros(2, **i32), out=out)
    assert bool((out == 5).all())
    q = torch.ones(1, 4, 64, **bf)
    assert bool((mol.mol_paged_attention(q, kc, kc, table[:, :0], lens) == 0).all())
    assert bool((mol.mol_paged_attention(q, kc[:0], kc[:0], table, lens) == 0).all())
