"""GPU tests of every way that paged attention takes through its kernels: the forms for few and for many
rows, in the release and the checked build, many sequences, long ones in hundreds of parts, strided
operands, caches past 32-bit offsets, waits that run out. The bounds: tests/attn_util.py."""

import numpy as np
import pytest

from tests import attn_util as au
from tests.gpu_util import mol_lib, torch_cuda
from tests.test_gpu_attn import attend, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return torch_cuda(), mol_lib()


@pytest.fixture(scope="module", params=["release", "checked"])
def build(request, env):
    """Both builds; the checked one records no failed check."""
    torch, mol = env
    if request.param == "release":
        yield env
        return
    from moe_lora_virtual_gb300.build import build_library

    with mol.use_library(build_library(checked=True)):
        mol.mol_take_check_record()
        yield env
        rec = mol.mol_take_check_record()
        assert rec.count == 0, f"{rec.count} failed checks, first {rec.site_name} value {rec.value}"
        assert mol.mol_take_fault_flags() == 0


# Rows a sequence on average (new tokens x group): up to 16, up to 32, more; with others among them.
FORMS = [([(1, 90)] * 5, 8, 2), ([(4, 90), (6, 700), (1, 3)], 8, 2), ([(6, 90), (5, 300), (30, 64)], 8, 2),
         ([(300, 300), (1, 40), (70, 900)], 8, 2), ([(129, 1000)], 3, 3), ([(64, 64), (63, 129)], 14, 2)]


@pytest.mark.parametrize("lens,Hq,Hkv", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page,order", [(16, "nhd"), (8, "hnd"), (64, "hnd"), (128, "nhd"), (256, "nhd"),
                                        (1, "nhd"), (48, "hnd")])
@pytest.mark.parametrize("window", [0, 50])
def test_forms(build, lens, Hq, Hkv, D, page, order, window):
    torch, _ = build
    run(build, au.problem(torch, D + page + window, lens, Hq, Hkv, D, page, order, lead=2, tail=1,
                          holes=0.1 if page < 64 else 0.0), window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("B,n,kv", [(129, 1, 20), (700, 1, 5), (400, 3, 9), (390, 20, 24), (130, 40, 70)])
def test_more_sequences_than_threads(build, D, B, n, kv):
    torch, _ = build
    rng = np.random.default_rng(B)
    lens = [(int(rng.integers(0, n + 1)) if n > 1 else 1, int(rng.integers(0, kv))) for _ in range(B)]
    lens = [(min(m, k) if n > 1 else m, k) for m, k in lens]
    run(build, au.problem(torch, B, lens, 4, 2, D, 16))


# --------------------------------------------------------------------- against float64 on the device
def exact(torch, p, scale, window=0):
    """(out, bound) on the device, sequence by sequence, without holes."""
    kc, vc = au.caches(p, "cuda")
    q, D = p["q"].cuda().double(), p["q"].shape[2]
    group = q.shape[1] // kc.shape[2]
    starts = list(range(len(p["kv_lens"]) + 1)) if p["starts"] is None else p["starts"].tolist()
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    for b, kv in enumerate(p["kv_lens"].tolist()):
        rows = slice(starts[b], starts[b + 1])
        n = starts[b + 1] - starts[b]
        pages = p["table"][b, :-(-kv // p["page"])].long().cuda()
        pos = torch.arange(kv - n, kv, device="cuda").unsqueeze(1)
        j = torch.arange(kv, device="cuda")
        sees = (j <= pos) & ((j > pos - window) if window else True)
        for h in range(kc.shape[2]):
            k, v = (t[pages, :, h].reshape(-1, D)[:kv].double() for t in (kc, vc))
            for i in range(h * group, (h + 1) * group):
                w = (scale * (q[rows, i] @ k.T)).masked_fill(~sees, -float("inf")).softmax(1)
                reach = (scale * (q[rows, i].abs() @ k.abs().T)).masked_fill(~sees, 0.0).amax(1)
                out[rows, i] = w @ v
                score = (D * 2.0 ** -24 + 2.0 ** -21) * reach.unsqueeze(1)
                bound[rows, i] = au.ROUND * out[rows, i].abs() + (
                    au.ROUND + 2 * score + 2.0 ** -13) * (w @ v.abs())
    return out, bound


def near(torch, got, p, scale, window=0):
    want, bound = exact(torch, p, scale, window)
    err = (got.cuda().double() - want).abs()
    bad = ~(err <= bound)
    assert not bool(bad.any()), (bad.nonzero()[:4].tolist(), err[bad][:4])


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,window", [
    ([(1, 40000)], 8, 1, 128, 16, 0),               # hundreds of parts of one head
    ([(1, 16000), (1, 1), (1, 9000)], 4, 2, 64, 32, 0), ([(1, 12000)], 2, 1, 256, 64, 0),
    ([(40, 30000)], 8, 1, 128, 16, 0), ([(33, 16000), (200, 9000)], 8, 2, 64, 64, 3000),
    ([(2048, 2048)], 4, 2, 128, 64, 0), ([(1000, 5000), (1, 7000), (37, 37)], 8, 4, 64, 16, 1024),
    ([(700, 3000)], 1, 1, 128, 128, 0), ([(300, 9000), (1, 77)], 4, 2, 256, 16, 0),
    ([(130, 5000), (700, 1400)], 3, 1, 256, 64, 900)])
def test_long(env, lens, Hq, Hkv, D, page, window):
    torch, _ = env
    p = au.problem(torch, D, lens, Hq, Hkv, D, page)
    near(torch, attend(env, p, window), p, D ** -0.5, window)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [0, 150])
@pytest.mark.parametrize("most", [3, 6, 90, 300])
def test_many_blocks_of_unlike_sizes(env, D, window, most):
    """A thread block goes through several blocks of rows, of one query tile and of two, of one tile of
    keys and of several, and through parts of some."""
    torch, _ = env
    rng = np.random.default_rng(D + window + most)
    lens = [(int(rng.integers(1, most + 1)), int(rng.integers(1, 1200))) for _ in range(150)]
    lens = [(min(n, kv), kv) for n, kv in lens]
    p = au.problem(torch, most, lens, 8, 4, D, 16)
    near(torch, attend(env, p, window), p, D ** -0.5, window)


@pytest.mark.parametrize("scale", [1e-4, 3.0])
@pytest.mark.parametrize("lens", [[(1, 3000)], [(200, 3000)]])
def test_flat_and_sharp_weights(env, scale, lens):
    """Scores near 0, and hundreds of powers of two apart, the largest anywhere in the sequence."""
    torch, _ = env
    for D in (64, 128, 256):
        p = au.problem(torch, D, lens, 4, 2, D, 16, std=3.0)
        near(torch, attend(env, p, scale=scale), p, scale)


def test_scores_that_rise_and_fall(env):
    """Maxima that grow from tile to tile (sums rescaled each time), and that only the first tile has."""
    torch, mol = env
    for D, lens in ((64, [(1, 1000)]), (128, [(150, 1000)]), (64, [(150, 1000)]),
                    (256, [(1, 1000)]), (256, [(150, 1000)])):
        p = au.problem(torch, D, lens, 4, 2, D, 16)
        k, _ = au.caches(p, "cpu")
        p["q"][..., 0] = 8.0
        for up in (1, -1):
            for i, page in enumerate(p["table"][0, :-(-1000 // 16)].tolist()):
                k[page, :, :, 0] = up * (i - 31.0)
            near(torch, attend(env, p, scale=0.5), p, 0.5)


@pytest.mark.parametrize("lens", [[(1, 50), (1, 90)], [(5, 50), (150, 200)]])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_strided_operands(env, lens, D):
    """Queries inside a joint projection's rows, outputs inside wider rows, heads before tokens, keys
    and values of a page in one buffer, a table inside a wider one."""
    torch, mol = env
    p = au.problem(torch, D, lens, 6, 2, D, 16)
    want = attend(env, p)
    T = p["q"].shape[0]
    joint = torch.full((T, 10, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    joint[:, 1:7] = p["q"].cuda()
    both = torch.stack([p["k"], p["v"]], 1).cuda()
    table = torch.full((len(lens), p["table"].shape[1] + 3), 1 << 30, dtype=torch.int32, device="cuda")
    table[:, :-3] = p["table"].cuda()
    starts = None if p["starts"] is None else p["starts"].cuda()
    wide = torch.full((T, 6, D + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    got = mol.mol_paged_attention(joint[:, 1:7], both[:, 0], both[:, 1], table[:, :-3], p["kv_lens"].cuda(),
                                  starts, out=wide[..., :D])
    assert torch.equal(got.cpu(), want) and bool((wide[..., D:] == 7).all())
    heads_first = p["q"].cuda().transpose(0, 1).contiguous().transpose(0, 1)
    out = torch.empty(6, T, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    kc, vc = au.caches(p, "cuda")
    mol.mol_paged_attention(heads_first, kc, vc, p["table"].cuda(), p["kv_lens"].cuda(), starts, out=out)
    assert torch.equal(out.cpu(), want)


@pytest.mark.parametrize("D,Hkv,page", [(128, 8, 64), (64, 4, 16)])
def test_past_32_bit_offsets(env, D, Hkv, page):
    """A cache of more than 2^31 values of which the last pages are used, appended to and read."""
    torch, mol = env
    pages = (1 << 31) // (page * Hkv * D) + 40
    kc, vc = (torch.empty(pages, page, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator().manual_seed(D)
    lens = [(1, 200), (1, 3 * page)]
    for counts in ([1, 1], [90, 40]):
        T = sum(counts)
        kv = [200, 3 * page]
        table = torch.full((2, 16), -1, dtype=torch.int32)
        ids = torch.arange(pages - 32, pages).flip(0).to(torch.int32)
        for b in range(2):
            n = -(-kv[b] // page)
            table[b, :n] = ids[16 * b:16 * b + n] if n <= 16 else ids[:n]
        small = au.problem(torch, D, list(zip(counts, kv)), 2 * Hkv, Hkv, D, page)
        sk, sv = au.caches(small, "cuda")
        rows, slots = [], []
        for b in range(2):
            for j in range(kv[b]):
                at = int(small["table"][b, j // page]), j % page
                rows.append(at)
                slots.append(int(table[b, j // page]) * page + j % page)
        i, o = (torch.tensor(x, device="cuda") for x in zip(*rows))
        mol.mol_cache_append(sk[i, o], sv[i, o], kc, vc, torch.tensor(slots, dtype=torch.int32, device="cuda"))
        starts = torch.tensor([0, counts[0], T], dtype=torch.int32, device="cuda")
        got = mol.mol_paged_attention(small["q"].cuda(), kc, vc, table.cuda(),
                                      torch.tensor(kv, dtype=torch.int32, device="cuda"), starts)
        # (a table of the same width: by that the host decides how blocks are dealt out)
        same = torch.full((2, 16), -1, dtype=torch.int32)
        same[:, :small["table"].shape[1]] = small["table"][:, :16]
        assert torch.equal(got.cpu(), attend(env, dict(small, starts=starts.cpu(), table=same)))


@pytest.mark.parametrize("page", [16, 5])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[(100, 300), (20, 700)], [(300, 300), (20, 700)]])
def test_wait_runs_out_sets_flag_then_device_recovers(env, D, page, lens):
    """With nothing copied every wait of the form for many rows gives up: the call returns, bit 0 is
    reported, nothing was written; the same call right after is right, with no bit set."""
    torch, mol = env
    p = au.problem(torch, D, lens, 4, 2, D, page)
    want = attend(env, p)
    assert mol.mol_take_fault_flags() == 0
    try:
        mol.mol_debug_wait_test(True, 2_000_000)  # waits give up after 2 ms
        got = attend(env, p, fill=7.0)
        flags = mol.mol_take_fault_flags()
    finally:
        mol.mol_debug_wait_test(False, 0)
    assert flags == 1 and bool((got == 7.0).all())
    assert torch.equal(attend(env, p), want) and mol.mol_take_fault_flags() == 0


def test_two_calls_at_once(env):
    """Calls on two streams, each with memory of its own, over one cache."""
    torch, mol = env
    p = au.problem(torch, 5, [(120, 4000), (1, 900)], 8, 2, 128, 16)
    want = attend(env, p).cuda()
    kc, vc = au.caches(p, "cuda")
    args = (p["q"].cuda(), kc, vc, p["table"].cuda(), p["kv_lens"].cuda(), p["starts"].cuda())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            outs[i].append(mol.mol_paged_attention(*args, stream=s))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for half in outs for o in half)


def test_two_graphs_with_one_workspace(env):
    """Replayed in turn, two captured calls may share their scratch."""
    torch, mol = env
    p = au.problem(torch, 6, [(1, 4000), (1, 900)], 8, 2, 128, 16)
    r = au.problem(torch, 7, [(130, 2000)], 8, 2, 64, 64)
    ws = torch.empty(max(mol.mol_paged_attention_workspace_bytes(2, 2, 8, 2, 128),
                         mol.mol_paged_attention_workspace_bytes(1, 130, 8, 2, 64)), dtype=torch.uint8,
                     device="cuda")
    graphs, outs, wants = [], [], []
    for x in (p, r):
        wants.append(attend(env, x).cuda())
        kc, vc = au.caches(x, "cuda")
        args = (x["q"].cuda(), kc, vc, x["table"].cuda(), x["kv_lens"].cuda(),
                None if x["starts"] is None else x["starts"].cuda())
        out = torch.empty_like(args[0])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mol.mol_paged_attention(*args, out=out, workspace=ws)
        graphs.append((graph, args))
        outs.append(out)
    for i in (0, 1, 1, 0, 1):
        outs[i].zero_()
        graphs[i][0].replay()
        assert torch.equal(outs[i], wants[i])
