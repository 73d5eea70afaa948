"""CPU checks of the sizes at which paged attention's 32-bit numbers end: the last ones that are taken and
the first ones that are not. A call without scratch is refused behind the sizes, so none reaches a kernel."""

import re

import pytest

from tests.test_abi_cpu import mol, needs_nvcc  # noqa: F401  (fixture)
from tests.test_attn_cpu import CAPACITY, P, UNSUPPORTED, cache, header

pytestmark = needs_nvcc


def attend(mol, T, H, B=1, pages=4, **c):  # noqa: F811
    """The status of a call whose sizes are as given and whose scratch is missing."""
    c = cache(**c)
    return mol.library().mol_paged_attention(
        P(16), 64 * H, 64, c, P(16), pages, pages, P(16), P(16), B, T, H, 0.125, 0, P(16), 64 * H, 64, None, 0, None)


@pytest.mark.parametrize("group", [2, 16, 64])
def test_rows_of_a_key_head(mol, group):  # noqa: F811
    """A sequence's rows are rounded up to blocks of up to 256 in 32 bits: past 2^31 - 256 of them that sum
    is below 0, and there would be no block. Taken up to 2^31 - 1024."""
    last = ((1 << 31) - 1024) // group
    one = dict(heads=1, ps=8 * 64, ts=64)
    assert attend(mol, last, group, **one) == CAPACITY
    for T in (last + 1, ((1 << 31) - 1) // group):
        assert attend(mol, T, group, **one) == UNSUPPORTED
    # (with more key heads the rows of each are fewer)
    assert attend(mol, ((1 << 31) - 1) // (2 * group), 2 * group, heads=2) == CAPACITY


def test_tiles_of_a_head(mol):  # noqa: F811
    """8 M cached tokens in pages of 8, group 8: the product of the header's bound passes 2^31 between 32765
    tokens and 32766."""
    for T, status in ((32765, CAPACITY), (32766, UNSUPPORTED), (32768, UNSUPPORTED)):
        assert attend(mol, T, 16, pages=1 << 20) == status
        assert ((T * 8 // 16 + 1) * ((8 << 20) // 64 + 4) < 1 << 31) == (status == CAPACITY)


def test_the_size_that_the_header_offers_is_taken(mol):  # noqa: F811
    offered = re.search(r"\((\d+) K (?:rows|tokens) of group (\d+) over\s+(?:\*\s+)?tables of (\d+) M", header())
    T, group, cached = (int(x) for x in offered.groups())
    assert attend(mol, T << 10, 2 * group, pages=cached << 17) == CAPACITY
