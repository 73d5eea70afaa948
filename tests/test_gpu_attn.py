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


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 1, 70, (1 << 31) - 1])
@pytest.mark.parametrize("lens", [[(5, 3), (4, 0), (1, 40)], [(400, 90), (300, 0), (5, 3), (70, 69)]])
def test_more_rows_than_cached_tokens(env, D, window, lens):
    """Rows before position 0 see nothing, whatever the window; those behind them what is there."""
    torch, _ = env
    got = run(env, au.problem(torch, D + window % 1000, lens, 8, 4, D, 16), window)
    for (n, kv), at in zip(lens, np.cumsum([0] + [n for n, _ in lens])):
        assert bool((got[at:at + max(n - kv, 0)] == 0).all())


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


# ------------------------------------------------------------------------------------ the calls
def step(torch, mol, g, T=5, Hq=4, Hkv=2, D=64, page=8, kv=40):
    """Tensors of one attention step of T sequences with a token each, and the calls on them."""
    pages = T * (kv // page) + 2
    s = dict(rows=randn(torch, g, T, Hq + 2 * Hkv, D).cuda(), rope=mol.rope_frequencies(32, device="cuda"),
             kc=randn(torch, g, pages, page, Hkv, D).cuda(), vc=randn(torch, g, pages, page, Hkv, D).cuda(),
             table=torch.randperm(pages, generator=g)[:T * (kv // page)].to(torch.int32).view(T, -1).cuda(),
             lens=torch.randint(1, kv + 1, (T,), generator=g).to(torch.int32).cuda())
    at = (s["lens"] - 1).long()
    s["positions"] = at.to(torch.int32)
    s["slots"] = (s["table"].gather(1, (at // page).unsqueeze(1)).view(-1) * page + at % page).to(torch.int32)

    def run(**kw):
        r = s["rows"]
        x = mol.mol_rope(r[:, :Hq], s["positions"], s["rope"], **kw)
        q = mol.mol_cache_append(r[:, Hq:Hq + Hkv], r[:, Hq + Hkv:], s["kc"], s["vc"], s["slots"],
                                 s["positions"], s["rope"], q=r[:, :Hq], **kw)
        out = mol.mol_paged_attention(q, s["kc"], s["vc"], s["table"], s["lens"], **kw)
        return x, q, out, s["kc"], s["vc"]

    return s, run


def test_native_calls_equal_the_python_path(env, monkeypatch):
    torch, mol = env
    from moe_lora_virtual_gb300 import block
    assert block._native is not None, "the native calls are not built"
    g = torch.Generator().manual_seed(2)
    s, run = step(torch, mol, g)
    taken, real = [], block._native

    class Count:
        def __getattr__(self, name):
            def call(*a):
                out = getattr(real, name)(*a)
                taken.append(out is not None)
                return out
            return call

    monkeypatch.setattr(block, "_native", Count())
    got = [t.clone() for t in run()]
    starts = torch.tensor([0, 2, 2, 3, 5, 5], dtype=torch.int32, device="cuda")
    more = mol.mol_paged_attention(got[1], s["kc"], s["vc"], s["table"], s["lens"], starts, scale=0.3, window=9)
    assert mol.mol_cache_append(s["rows"][:, :2], s["rows"][:, 2:4], s["kc"], s["vc"], s["slots"]) is None
    plain = [s["kc"].clone(), s["vc"].clone()]
    assert len(taken) == 5 and all(taken)
    monkeypatch.setattr(block, "_native", None)
    mol.mol_cache_append(s["rows"][:, :2], s["rows"][:, 2:4], s["kc"], s["vc"], s["slots"])
    assert torch.equal(plain[0], s["kc"]) and torch.equal(plain[1], s["vc"])
    for a, b in zip(got, run()):
        assert torch.equal(a, b)
    assert torch.equal(more, mol.mol_paged_attention(got[1], s["kc"], s["vc"], s["table"], s["lens"], starts,
                                                     scale=0.3, window=9))


def test_a_layer_step_in_a_graph_and_on_a_stream(env):
    """The three calls as a decoding step makes them: captured and replayed on new rows and lengths, and
    on a stream of their own."""
    torch, mol = env
    g = torch.Generator().manual_seed(3)
    s, run = step(torch, mol, g, T=9, D=128, kv=96)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run()
    s["rows"].copy_(randn(torch, g, *s["rows"].shape))
    fresh = torch.randint(1, 97, (9,), generator=g).to(torch.int32).cuda()
    s["lens"].copy_(fresh)
    kc, vc = s["kc"].clone(), s["vc"].clone()
    graph.replay()
    got = [t.clone() for t in captured]
    s["kc"].copy_(kc), s["vc"].copy_(vc)
    for a, b in zip(got, run()):
        assert torch.equal(a, b)
    s["kc"].copy_(kc), s["vc"].copy_(vc)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = run(stream=side)
    side.synchronize()
    for a, b in zip(got, out):
        assert torch.equal(a, b)


@pytest.mark.parametrize("D,lens", [(64, [(1, 900), (1, 3)]), (128, [(200, 700), (1, 2000), (3, 9)]),
                                    (256, [(5, 1500)]), (256, [(200, 700), (1, 2000)])])
def test_results_do_not_depend_on_timing_or_what_memory_held(env, D, lens):
    """Bit-equal over calls, over workspaces of NaN and of ones, with the workspace of another size."""
    torch, mol = env
    p = au.problem(torch, D, lens, 8, 2, D, 16)
    first = attend(env, p)
    size = mol.mol_paged_attention_workspace_bytes(len(lens), p["q"].shape[0], 8, 2, D)
    for byte, more in ((0xFF, 0), (1, 4096), (0x7F, 16)):
        ws = torch.full((size + more,), byte, dtype=torch.uint8, device="cuda")
        assert torch.equal(attend(env, p, workspace=ws), first)


def test_out_may_be_the_queries(env):
    torch, mol = env
    for lens in ([(1, 70), (1, 2)], [(150, 150), (40, 700)]):
        p = au.problem(torch, 7, lens, 8, 2, 64, 16)
        want = attend(env, p)
        kc, vc = au.caches(p, "cuda")
        q = p["q"].cuda()
        got = mol.mol_paged_attention(q, kc, vc, p["table"].cuda(), p["kv_lens"].cuda(),
                                      None if p["starts"] is None else p["starts"].cuda(), out=q)
        assert got is q and torch.equal(got.cpu(), want)


def test_binding_refusals(env):
    torch, mol = env
    bf, i32 = (dict(dtype=d, device="cuda") for d in (torch.bfloat16, torch.int32))
    x, pos = torch.zeros(3, 4, 64, **bf), torch.zeros(3, **i32)
    kc, vc = torch.zeros(2, 8, 2, 64, **bf), torch.zeros(2, 8, 2, 64, **bf)
    k, rope = x[:, :2], mol.rope_frequencies(64, device="cuda")
    table, lens = torch.zeros(3, 2, **i32), torch.ones(3, **i32)
    wrong = [
        (ValueError, lambda: mol.mol_rope(x[0], pos, rope)),
        (ValueError, lambda: mol.mol_rope(x, pos[:2], rope)),
        (TypeError, lambda: mol.mol_rope(x, pos.long(), rope)),
        (TypeError, lambda: mol.mol_rope(x.float(), pos, rope)),
        (TypeError, lambda: mol.mol_rope(x.cpu(), pos, rope)),
        (ValueError, lambda: mol.mol_rope(x.transpose(1, 2), pos, rope)),
        (mol.MolError, lambda: mol.mol_rope(x[..., :32], pos, rope)),
        (ValueError, lambda: mol.mol_rope(x, pos, rope, out=x[:, :2])),
        (ValueError, lambda: mol.mol_cache_append(x, x, kc, vc, pos)),
        (ValueError, lambda: mol.mol_cache_append(k, k[:2], kc, vc, pos)),
        (ValueError, lambda: mol.mol_cache_append(k, k, kc, vc[:1], pos)),
        (ValueError, lambda: mol.mol_cache_append(k, k, kc, vc, pos, rope=rope)),
        (ValueError, lambda: mol.mol_cache_append(k, k, kc, vc, pos, q=x)),
        (ValueError, lambda: mol.mol_cache_append(k, k, kc, vc, pos, pos, rope, q_out=x)),
        (ValueError, lambda: mol.mol_cache_append(k, k, kc, vc, pos, pos, rope, q=x[:2])),
        (ValueError, lambda: mol.mol_cache_append(k, k, kc, torch.zeros(2, 2, 8, 64, **bf).transpose(1, 2), pos)),
        (ValueError, lambda: mol.mol_paged_attention(x[:2], kc, vc, table, lens)),
        (ValueError, lambda: mol.mol_paged_attention(x, kc, vc, table[0], lens)),
        (ValueError, lambda: mol.mol_paged_attention(x, kc, vc, table, lens[:2])),
        (ValueError, lambda: mol.mol_paged_attention(x, kc, vc, table, lens, pos)),
        (ValueError, lambda: mol.mol_paged_attention(x[..., :32], kc, vc, table, lens)),
        (TypeError, lambda: mol.mol_paged_attention(x, kc, vc, table.long(), lens)),
        (ValueError, lambda: mol.mol_paged_attention(x, kc, vc, table.t(), lens[:2], pos)),
        (mol.MolError, lambda: mol.mol_paged_attention(x[:, :3], kc, vc, table, lens)),
        (mol.MolError, lambda: mol.mol_paged_attention(x, kc, vc, table, lens, scale=0.0)),
        (mol.MolError, lambda: mol.mol_paged_attention(x, kc, vc, table, lens, window=-1)),
        (mol.MolError, lambda: mol.mol_paged_attention(x, kc, vc, table, lens,
                                                       workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))),
    ]
    for i, (error, call) in enumerate(wrong):
        with pytest.raises(error):
            call()
            pytest.fail(f"call {i} was taken")


def example():
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decode_layers.py")
    spec = importlib.util.spec_from_file_location("decode_layers", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_example_attention_half(env):
    """The example's attention over a prompt and the tokens behind it against the same in float64, with
    bf16 where the layer holds bf16: the norm, the projection, the cache's keys and the queries, the
    weights, the attention and the output are seven roundings in a row of 2^-8 each, taken in the mean
    square over the rows."""
    torch, mol = env
    module = example()
    g = torch.Generator(device="cuda").manual_seed(1)
    H, heads, kv, D = 256, 8, 2, 64
    batch = module.Batch(3, 200, 16)
    half = module.Attention(g, H, heads, kv, D, batch, 64)
    x = torch.randn(64, H, generator=g, device="cuda").to(torch.bfloat16)
    zero = torch.zeros_like(x)
    chunks = [[30, 0, 14], [1, 20, 3], None, [0, 2, 1], None]
    rows, seen, want, got = 0, [[], [], []], [], []
    qkv, proj = mol.w4_unpack(half.qkv).double(), mol.w4_unpack(half.out).double()
    for counts in chunks:
        n = 3 if counts is None else sum(counts)
        here = x[rows:rows + n] if rows + n <= len(x) else x[:n]
        place = batch.place(counts)
        y, _ = half(zero[:n], here, batch, place)
        got.append(y.clone())
        r = here.double()
        normed = r * torch.rsqrt((r * r).mean(-1, keepdim=True) + 1e-6)
        p = (normed @ qkv.T).view(n, -1, D).cpu().numpy()
        freq = f64(half.rope.inv_freq)
        at = f64(place[0])
        q, k = ao.rope(p[:, :heads], at, freq), ao.rope(p[:, heads:heads + kv], at, freq)
        row = 0
        for b, m in enumerate([1, 1, 1] if counts is None else counts):
            for _ in range(m):
                assert at[row] == len(seen[b])
                seen[b].append((k[row], p[row, heads + kv:]))
                ks, vs = (np.stack([t[i] for t in seen[b]]) for i in (0, 1))
                s = np.einsum("hd,jhd->hj", q[row], np.repeat(ks, heads // kv, 1)) * D ** -0.5
                w = np.exp(s - s.max(1, keepdims=True))
                o = np.einsum("hj,jhd->hd", w / w.sum(1, keepdims=True), np.repeat(vs, heads // kv, 1))
                want.append(o.reshape(-1) @ proj.cpu().numpy().T)
                row += 1
        rows = (rows + n) % 40
    got, want = f64(torch.cat(got)), np.stack(want)
    err = np.sqrt(((got - want) ** 2).mean() / (want ** 2).mean())
    assert err < 7 ** 0.5 * ROUND, err


def test_example_model_with_attention_in_a_graph(env):
    """Steps of the whole model, a prompt first: the replayed graph gives what the calls give."""
    torch, mol = env
    module = example()
    T = 5
    kw = dict(tokens=T, layers=2, group=0, seed=3, heads=4, kv_heads=2, head_dim=64, context=64, page=8)
    g = torch.Generator().manual_seed(4)
    prompt = torch.randint(0, 5000, (17,), generator=g).cuda()
    tokens = torch.randint(0, 5000, (3, T), generator=g).cuda()
    lora = torch.randint(-1, 4, (17,), generator=g).to(torch.int32).cuda()
    # (as many pairs as the model's buffers hold: five tokens at a time)
    parts = [[2, 1, 0, 1, 1], [0, 3, 1, 0, 1], [5, 0, 0, 0, 0]]

    def begin():
        torch.manual_seed(7)  # the pages' order
        model, at = module.Model(**kw), 0
        for counts in parts:
            model(prompt[at:at + sum(counts)], lora[at:at + sum(counts)], counts)
            at += sum(counts)
        return model

    model = begin()
    want = [model(t, lora[:T]).clone() for t in tokens]
    assert model.batch.lens.tolist() == [10, 7, 4, 4, 5]
    model = begin()
    first = model(tokens[0], lora[:T])  # (before the capture, on the same cache)
    assert torch.equal(first, want[0])
    step = tokens[1].clone()
    graph = torch.cuda.CUDAGraph()
    lens = model.batch.lens.clone()
    with torch.cuda.graph(graph):
        logits = model(step, lora[:T])
    assert torch.equal(model.batch.lens, lens)
    for i in (1, 2):
        step.copy_(tokens[i])
        graph.replay()
        assert torch.equal(logits, want[i])
