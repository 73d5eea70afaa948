"""GPU tests of paged attention's sums over millions of cached tokens by one thread block.

Queries of 0 give every token the same weight, 1 before the division, in bf16 as in fp32, and values between 1
and 2 a sum that grows with every token. What an output may be off by is then its own rounding, 2^-8, and
what the sums lose: matrix instructions add 16 tokens to an fp32 sum and cut what does not fit it, twice 2^-23
of it at most. The kernels let such a sum run over 2^16 tokens, 2^12 instructions of a warp or a tensor core:
2^-10. (Without that the outputs here are 1 % off.)
"""

import pytest

from tests import attn_util as au
from tests.gpu_util import mol_lib, torch_cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def env():
    return torch_cuda(), mol_lib()


# (sequences, new tokens each, log2 of the cached tokens): blocks of 16 rows and of 32, one or two for each of
# 304 thread blocks (152 for 256 values a head), whose four warps share the tokens; blocks of many rows
@pytest.mark.parametrize("B,n,kv,D,page", [
    (608, 1, 23, 64, 128), (608, 1, 23, 128, 128), (304, 1, 23, 256, 128), (304, 17, 23, 64, 128),
    (1, 256 * 152, 21, 64, 128), (152, 100, 21, 64, 128), (1, 256 * 152, 21, 128, 128), (1, 256 * 152, 21, 128, 120),
    (1, 128 * 152, 21, 256, 128)])
@pytest.mark.parametrize("rises", [0, 1])
def test_flat_weights_over_long_contexts(env, B, n, kv, D, page, rises):
    """rises: the scores of the last tokens are larger by a power of two or so, so that sums are brought to
    another maximum after they were put aside; their weights are powers of two and exact."""
    torch, mol = env
    kv = 1 << kv
    g = torch.Generator(device="cuda").manual_seed(D)
    pages = -(-kv // page)
    k = torch.zeros(pages, page, 1, D, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    for i in range(0, pages, 1 << 12):
        v[i:i + (1 << 12)] = torch.rand(v[i:i + (1 << 12)].shape, generator=g, device="cuda") + 1
    flat_k, flat_v = k.view(-1, D), v.view(-1, D)
    # the last 2^18 tokens before the new ones: weights of 2^12
    late = kv - n - (1 << 18)
    if rises:
        flat_k[late:, 0] = 1.0
    q = torch.zeros(B * n, 1, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 12.0  # (times log2(e) below: a power of two a unit)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()
    lens = torch.full((B,), kv, dtype=torch.int32, device="cuda")
    starts = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    got = mol.mol_paged_attention(q, k, v, table, lens, starts, scale=0.6931471805599453)

    early = torch.zeros(D, dtype=torch.float64, device="cuda")
    for i in range(0, late, 1 << 20):
        early += flat_v[i:min(late, i + (1 << 20))].double().sum(0)
    weight = 4096.0 if rises else 1.0
    rows = late + torch.arange(1, kv - late + 1, device="cuda")  # (the token count of a row at each late token)
    sums = early + weight * flat_v[late:kv].double().cumsum(0)
    want = (sums / (late + weight * (rows - late)).unsqueeze(1))[-n:]
    err = (got.view(B, n, D).double() - want).abs() / want
    assert float(err.max()) <= 2.0 ** -8 + 2.0 ** -10, float(err.max())


# Sequences of unlike lengths over one cache, so many that a thread block goes through whole ones of several
# stretches, and through parts of them: few rows (16, 32), many, 256 values a head; a window of several stretches
@pytest.mark.parametrize("B,n,D,Hkv,group,page,window", [
    (300, 1, 64, 2, 4, 64, 0), (300, 1, 128, 2, 4, 64, 0), (150, 1, 256, 2, 4, 64, 0), (150, 5, 64, 2, 5, 64, 0),
    (150, 1, 128, 2, 4, 64, 100000), (80, 64, 64, 2, 8, 64, 0), (80, 64, 64, 2, 8, 64, 140000),
    (80, 64, 128, 2, 8, 64, 0), (80, 64, 128, 2, 8, 40, 0), (160, 11, 128, 2, 3, 64, 90000), (80, 33, 256, 2, 4, 64, 0),
    (80, 33, 256, 2, 4, 64, 100000)])
def test_stretches_join(env, B, n, D, Hkv, group, page, window):
    """Against float64, with holes among the pages."""
    torch, mol = env
    longest = 200000
    whole = au.problem(torch, D, [(n, longest)], Hkv * group, Hkv, D, page, holes=0.02)
    kc, vc = au.caches(whole, "cuda")
    g = torch.Generator().manual_seed(B)
    lens = [longest - 100] + torch.randint(66000, longest, (B - 1,), generator=g).tolist()
    q = (torch.randn(B * n, Hkv * group, D, generator=g) * 1.5).to(torch.bfloat16).cuda()
    table = whole["table"].expand(B, -1).contiguous().cuda()
    starts = None if n == 1 else torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    scale = D ** -0.5
    out = mol.mol_paged_attention(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), starts,
                                  window=window)
    again = mol.mol_paged_attention(q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), starts,
                                    window=window)
    assert torch.equal(out, again)
    held = ((whole["table"][0] >= 0) & (whole["table"][0] < kc.shape[0])).cuda()
    seen = held.repeat_interleave(page)[:longest]
    pages = whole["table"][0].clamp(0, kc.shape[0] - 1).long().cuda()
    for h in range(Hkv):
        k, v = (torch.where(seen.unsqueeze(1), t[pages, :, h].reshape(-1, D)[:longest].double(), 0.0)
                for t in (kc, vc))
        for b in {0, 1, 2, B // 3, B // 2, B - 2, B - 1}:
            kv, rows = lens[b], q[b * n:(b + 1) * n, h * group:(h + 1) * group].double()
            pos = torch.arange(kv - n, kv, device="cuda").view(n, 1, 1)
            j = torch.arange(kv, device="cuda")
            sees = (j <= pos) & seen[:kv]
            if window:
                sees &= j > pos - window
            x = (rows @ k[:kv].T * scale).masked_fill(~sees, -float("inf"))
            w = x.softmax(2)
            reach = (rows.abs() @ k[:kv].abs().T * scale).masked_fill(~sees, 0.0).amax(2, keepdim=True)
            want, spread = w @ v[:kv], w @ v[:kv].abs()
            score = (D * 2.0 ** -24 + 2.0 ** -21) * reach
            # (sums cut as above, 2^-10, for the 2^-13 of shorter ones)
            bound = au.ROUND * want.abs() + (au.ROUND + 2 * score + 2.0 ** -10) * spread
            err = (out[b * n:(b + 1) * n, h * group:(h + 1) * group].double() - want).abs()
            bad = ~(err <= bound)
            assert not bool(bad.any()), (b, h, bad.nonzero()[:4].tolist(), err[bad][:4])
