"""Numbers of the attention half's calls that 32 bits do not hold: the C calls take int32, and ctypes keeps
the low half of what is larger."""

import pytest

from tests.test_abi_cpu import mol as library, needs_nvcc  # noqa: F401  (fixture)
from tests.test_block_binding_cpu import Stream, binding, cuda  # noqa: F401  (fixture)

torch = pytest.importorskip("torch")
import moe_lora_virtual_gb300 as mol  # noqa: E402

i32 = torch.int32
LAST = (1 << 31) - 1
WINDOW = 13  # its place among mol_paged_attention's arguments


@pytest.fixture
def handed(binding, monkeypatch):  # noqa: F811
    from moe_lora_virtual_gb300 import attention
    monkeypatch.setattr(attention, "mol_paged_attention_workspace_bytes", lambda *a: 4096)
    return binding.calls


def attend(**kw):
    q, kc = cuda(3, 4, 64), cuda(2, 8, 2, 64)
    mol.mol_paged_attention(q, kc, kc, cuda(3, 1, dtype=i32), cuda(3, dtype=i32), stream=Stream(0x10), **kw)


@pytest.mark.parametrize("window,at", [
    (0, 0), (5, 5), (LAST, LAST), (LAST + 1, LAST), (1 << 32, LAST), ((1 << 32) + 5, LAST), (1 << 70, LAST),
    (-1, -1), (5 - (1 << 32), -1 - LAST), (-(1 << 32), -1 - LAST)])
def test_a_window_past_32_bits_is_the_widest_there_is(handed, window, at):
    """All cached tokens lie within 2^31 - 1 of each other; one below 0 stays so, for the call to refuse."""
    attend(window=window)
    name, a = handed[-1]
    assert name == "mol_paged_attention" and a[WINDOW] == at


@pytest.mark.parametrize("window", [5.0, "5", None])
def test_a_window_that_is_no_integer_is_refused(handed, window):
    with pytest.raises(TypeError):
        attend(window=window)
    assert not handed


def test_sizes_past_32_bits_are_not_cut(handed):
    """Neither a cache's sizes (its strides of 0 are for the call to refuse) nor a layout that is none."""
    wide = cuda(1, 1, 2, 64).expand(1, (1 << 32) + 1, 2, 64)
    rows, at = cuda(3, 2, 64), cuda(3, dtype=i32)
    mol.mol_cache_append(rows, rows, wide, wide, at, stream=Stream(0x10))
    assert handed[-1][1][10].page_size == LAST
    mol.mol_rope(rows, at, mol.Rope(cuda(32, dtype=torch.float32), 1 << 32), stream=Stream(0x10))
    assert handed[-1][1][4].interleaved == LAST


@needs_nvcc
@pytest.mark.parametrize("at", [2, 3, 4])
def test_the_scratch_of_sizes_past_32_bits(library, at):  # noqa: F811
    sizes = [1, 1, 8, 2, 64]
    assert library.mol_paged_attention_workspace_bytes(*sizes) > 0
    sizes[at] += 1 << 32
    assert library.mol_paged_attention_workspace_bytes(*sizes) == 0
