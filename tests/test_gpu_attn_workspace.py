"""GPU tests of paged attention's scratch: nothing is written outside the least that a call accepts."""

import pytest

from tests import attn_util as au
from tests.gpu_util import mol_lib, torch_cuda
from tests.test_attn_cpu import CAPACITY
from tests.test_attn_workspace_cpu import attend as status
from tests.test_gpu_attn import attend

pytestmark = pytest.mark.gpu

GUARD = 1 << 20


@pytest.fixture(scope="module")
def env():
    return torch_cuda(), mol_lib()


def least(mol, B, T, group, D):
    """The fewest bytes that the call takes (asked with scratch that is not aligned, so that nothing runs)."""
    lo, hi = 0, mol.mol_paged_attention_workspace_bytes(B, T, group, 1, D)
    while hi - lo > 1:
        mid = (lo + hi) // 2
        lo, hi = (mid, hi) if status(mol, B, T, group, D, mid) == CAPACITY else (lo, mid)
    return hi


# Blocks in parts on every thread block of the launch: few rows (16 and 32 of them), many, 256 values a head;
# groups that do not divide a tile's 128 rows.
@pytest.mark.parametrize("lens,Hq,Hkv,D", [
    ([(1, 9000), (1, 5000), (1, 3)], 5, 1, 64), ([(1, 9000), (1, 5000), (1, 3)], 10, 2, 128),
    ([(1, 9000), (1, 5000), (1, 3)], 5, 1, 256), ([(6, 9000), (5, 5000), (6, 30)], 10, 2, 64),
    ([(300, 3000), (40, 5000), (1, 3)], 5, 1, 64), ([(300, 3000), (40, 5000), (1, 3)], 43, 1, 64),
    ([(300, 3000), (40, 5000), (1, 3)], 5, 1, 128), ([(300, 3000), (40, 5000), (1, 3)], 43, 1, 128),
    ([(300, 3000), (40, 5000), (1, 3)], 5, 1, 256), ([(300, 3000), (40, 5000), (1, 3)], 43, 1, 256)])
@pytest.mark.parametrize("page", [16, 5])
def test_nothing_outside_the_workspace_is_written(env, lens, Hq, Hkv, D, page):
    torch, mol = env
    p = au.problem(torch, D + Hq, lens, Hq, Hkv, D, page)
    size = least(mol, len(lens), p["q"].shape[0], Hq // Hkv, D)
    want = attend(env, p)
    room = torch.full((GUARD + -(-size // 16) * 16 + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    assert torch.equal(attend(env, p, workspace=room[GUARD:GUARD + size]), want)
    assert bool((room[:GUARD] == 0x5A).all()) and bool((room[GUARD + size:] == 0x5A).all())
    assert not bool((room[GUARD:GUARD + size] == 0x5A).all())  # (parts there were)
