"""GPU tests of paged attention whose lengths the kernel directly before writes, at its very end.

Calls whose blocks go undivided deal their rows from the lengths that memory holds while that kernel still
runs, and again where these turn out to have changed. The kernel before is a rotation of one token, which
releases its dependents at its beginning, goes through thousands of heads in one thread block, and copies the
fresh lengths, among the values of its last heads that are not turned, when it comes to them.
"""

import pytest

from tests import attn_util as au
from tests.gpu_util import mol_lib, torch_cuda

pytestmark = pytest.mark.gpu

HEADS = 4096


@pytest.fixture(scope="module")
def env():
    return torch_cuda(), mol_lib()


class Late:
    """Two int32 arrays, lengths and starts, and the call that writes them."""

    def __init__(self, torch, mol, lens, starts):
        self.x = torch.zeros(1, HEADS, 64, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros_like(self.x)
        self.fresh, self.arrays = [], []
        for head, values in ((-1, lens), (-2, starts)):
            assert len(values) <= 24
            for t, to in ((self.x, self.fresh), (self.out, self.arrays)):
                to.append(t[0, head, 16:].view(torch.int32)[:len(values)])
            self.fresh[-1].copy_(torch.tensor(values, dtype=torch.int32))
        rope, at = mol.rope_frequencies(16, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.write = lambda: mol.mol_rope(self.x, at, rope, out=self.out)

    def stale(self, torch, lens, starts):
        for t, values in zip(self.arrays, (lens, starts)):
            t.copy_(torch.tensor(values, dtype=torch.int32))


# (new tokens, cached tokens) of each sequence, fresh and before; D, query and key heads, page: undivided
# calls in blocks of 16 rows, of 32, of many (tensor copies, gathered tokens), of 256 values a head
CASES = [
    ([(1, 40), (1, 256), (1, 7), (1, 0)], [(1, 9), (1, 3), (1, 250), (1, 70)], 64, 8, 2, 16),
    ([(1, 40), (1, 130), (1, 7), (1, 0)], [(1, 9), (1, 3), (1, 120), (1, 70)], 128, 8, 2, 16),
    ([(1, 40), (1, 100), (1, 7), (1, 0)], [(1, 9), (1, 3), (1, 90), (1, 70)], 256, 8, 2, 16),
    ([(2, 40), (3, 200), (4, 7)], [(1, 9), (8, 60), (0, 140)], 64, 8, 2, 16),
    ([(6, 40), (7, 200), (2, 70)], [(1, 9), (8, 60), (6, 140)], 64, 8, 2, 16),
    ([(60, 90), (7, 200), (33, 400)], [(1, 9), (98, 160), (1, 440)], 64, 8, 2, 16),
    ([(160, 190), (7, 200), (133, 400)], [(1, 9), (298, 460), (1, 40)], 64, 8, 2, 16),
    ([(60, 90), (7, 200), (33, 400)], [(1, 9), (98, 160), (1, 440)], 64, 8, 2, 5),
    ([(60, 90), (7, 200), (33, 400)], [(1, 9), (98, 160), (1, 440)], 128, 8, 2, 16),
    ([(60, 90), (7, 200), (33, 400)], [(1, 9), (98, 160), (1, 440)], 128, 8, 2, 5),
    ([(60, 90), (7, 100), (33, 130)], [(1, 9), (98, 125), (1, 90)], 256, 8, 2, 16)]


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("now,before,D,Hq,Hkv,page", CASES)
def test_lengths_from_the_kernel_before(env, now, before, D, Hq, Hkv, page, captured):
    torch, mol = env
    widest = [(n, max(kv, was)) for (n, kv), (_, was) in zip(now, before)]
    p = au.problem(torch, D + page, widest, Hq, Hkv, D, page)
    lens, old = ([kv for _, kv in x] for x in (now, before))
    starts, was = ([sum(n for n, _ in x[:i]) for i in range(len(x) + 1)] for x in (now, before))
    p["kv_lens"] = torch.tensor(lens, dtype=torch.int32)
    want = au.oracle(p, D ** -0.5)
    kc, vc = au.caches(p, "cuda")
    q, table = p["q"].cuda(), p["table"].cuda()
    ws = torch.empty(mol.mol_paged_attention_workspace_bytes(len(lens), len(q), Hq, Hkv, D), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty_like(q)
    late = Late(torch, mol, lens, starts)

    def calls():
        late.write()
        mol.mol_paged_attention(q, kc, vc, table, late.arrays[0], None if p["starts"] is None else late.arrays[1],
                                out=out, workspace=ws)

    late.stale(torch, old, was)
    calls()  # (the library's kernels are prepared)
    run = calls
    if captured:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            calls()
        run = graph.replay
    for _ in range(3):
        late.stale(torch, old, was)
        out.fill_(9.0)
        torch.cuda.synchronize()
        run()
        torch.cuda.synchronize()
        assert late.arrays[0].tolist() == lens and late.arrays[1].tolist() == starts
        au.check(out.cpu(), *want)
