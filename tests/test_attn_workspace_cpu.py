"""CPU checks of the size query of paged attention's scratch: scratch of the size for some sequences and tokens
serves every call of at most so many, whatever form these take. (The scratch here is not aligned, which the
calls refuse behind their look at its size.)"""

import itertools

import pytest

from tests.test_abi_cpu import mol, needs_nvcc  # noqa: F401  (fixture)
from tests.test_attn_cpu import CAPACITY, P, UNSUPPORTED, cache

pytestmark = needs_nvcc

# (rows up to 16 a sequence, 32, more, with groups of 1 to 64)
SIZES = (1, 2, 3, 4, 5, 8, 9, 16, 17, 32, 33, 64, 65, 256, 257, 1000)


def attend(mol, B, T, group, D, ws):  # noqa: F811
    c = cache(D=D, hs=D, ts=2 * D, ps=16 * D)
    H = 2 * group
    return mol.library().mol_paged_attention(P(16), D * H, D, c, P(16), 4, 4, P(16), P(16), B, T, H, 0.125, 0, P(16),
                                             D * H, D, P(8), ws, None)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 4, 5, 16, 43, 64])
def test_scratch_of_the_largest_sizes_serves_the_others(mol, D, group):  # noqa: F811
    def size(B, T):
        return mol.mol_paged_attention_workspace_bytes(B, T, 2 * group, 2, D)

    for B, T in itertools.product(SIZES, SIZES):
        most = size(B, T)
        assert 0 < most < 128 << 20
        for b, t in itertools.product(SIZES, SIZES):
            if b <= B and t <= T:
                assert size(b, t) <= most
                assert attend(mol, b, t, group, D, most) == UNSUPPORTED, (B, T, b, t)
        assert attend(mol, B, T, group, D, 4096) == CAPACITY


def test_scratch_sized_for_one_call_still_serves_it(mol):  # noqa: F811
    """What the size was before it covered smaller calls: of 304 thread blocks two parts of 16 rows."""
    few = 304 * 2 * 16 * (128 * 4 + 8) + 304 * 32
    assert attend(mol, 256, 256, 8, 128, few) == UNSUPPORTED
    assert attend(mol, 1, 64, 8, 128, few) == CAPACITY


def test_no_scratch_for_sizes_that_are_refused(mol):  # noqa: F811
    size = mol.mol_paged_attention_workspace_bytes
    assert size(1, 1, 2 * 65, 2, 64) == 0 and size(1, 1, 2 * 64, 2, 64) > 0
