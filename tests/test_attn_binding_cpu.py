"""The Python path of the attention half's binding without a GPU (the stand-ins of
test_block_binding_cpu): what a call allocates where, and what it hands over."""

import pytest

from tests.test_block_binding_cpu import Cuda, Stream, binding, cuda  # noqa: F401  (fixture)

torch = pytest.importorskip("torch")
import moe_lora_virtual_gb300 as mol  # noqa: E402

i32, f32 = torch.int32, torch.float32


@pytest.fixture(autouse=True)
def sizes(binding, monkeypatch):  # noqa: F811
    from moe_lora_virtual_gb300 import attention
    monkeypatch.setattr(attention, "mol_paged_attention_workspace_bytes", lambda *a: 4096)


def calls(stream):
    """Every call with nothing passed in that it would allocate, and what it allocates."""
    T, Hq, Hkv, D, page = 5, 4, 2, 64, 8
    q, k = cuda(T, Hq, D), cuda(T, Hkv, D)
    caches = cuda(3, page, Hkv, D), cuda(3, page, Hkv, D)
    at = cuda(T, dtype=i32)
    rope = mol.Rope(cuda(D // 2, dtype=f32))
    return {
        "rope": (lambda: mol.mol_rope(q, at, rope, stream=stream), 1),
        "append": (lambda: mol.mol_cache_append(k, k, *caches, at, stream=stream), 0),
        "append with queries": (lambda: mol.mol_cache_append(k, k, *caches, at, at, rope, q=q, stream=stream), 1),
        "attention": (lambda: mol.mol_paged_attention(q, *caches, cuda(T, 2, dtype=i32), at, stream=stream), 2),
        "chunks": (lambda: mol.mol_paged_attention(q, *caches, cuda(2, 2, dtype=i32), at[:2].clone(),
                                                   cuda(3, dtype=i32), stream=stream), 2),
    }


@pytest.mark.parametrize("name", list(calls(None)))
def test_outputs_and_scratch_are_the_streams_own(binding, name):  # noqa: F811
    side = Stream(0x1230)
    call, tensors = calls(side)[name]
    binding.made.clear()
    call()
    assert len(binding.made) == tensors
    assert all(at is side for at, _ in binding.made), binding.made
    assert binding.calls[-1][1][-1] == 0x1230 and binding.at is None


@pytest.mark.parametrize("name", list(calls(None)))
def test_without_a_stream_the_current_one_is_used(binding, name, monkeypatch):  # noqa: F811
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0x77)
    call, tensors = calls(None)[name]
    binding.made.clear()
    call()
    assert [at for at, _ in binding.made] == [None] * tensors
    assert binding.calls[-1][1][-1] == 0x77


def moved(t):
    t = t.clone()
    t.on = 1
    return t


def test_operands_on_another_device_are_refused(binding):  # noqa: F811
    q, k, at = cuda(3, 4, 64), cuda(3, 2, 64), cuda(3, dtype=i32)
    c, table, rope = cuda(2, 8, 2, 64), cuda(3, 1, dtype=i32), mol.Rope(cuda(32, dtype=f32))
    side = Stream(0x10)
    wrong = [
        lambda: mol.mol_rope(moved(q), at, rope, stream=side),
        lambda: mol.mol_rope(q, moved(at), rope, stream=side),
        lambda: mol.mol_rope(q, at, mol.Rope(moved(rope.inv_freq)), stream=side),
        lambda: mol.mol_rope(q, at, rope, out=moved(q), stream=side),
        lambda: mol.mol_cache_append(moved(k), k, c, c, at, stream=side),
        lambda: mol.mol_cache_append(k, moved(k), c, c, at, stream=side),
        lambda: mol.mol_cache_append(k, k, moved(c), c, at, stream=side),
        lambda: mol.mol_cache_append(k, k, c, moved(c), at, stream=side),
        lambda: mol.mol_cache_append(k, k, c, c, moved(at), stream=side),
        lambda: mol.mol_cache_append(k, k, c, c, at, at, rope, q=moved(q), stream=side),
        lambda: mol.mol_paged_attention(moved(q), c, c, table, at, stream=side),
        lambda: mol.mol_paged_attention(q, moved(c), c, table, at, stream=side),
        lambda: mol.mol_paged_attention(q, c, c, moved(table), at, stream=side),
        lambda: mol.mol_paged_attention(q, c, c, table, moved(at), stream=side),
        lambda: mol.mol_paged_attention(q, c, c, table, at, moved(cuda(4, dtype=i32)), stream=side),
        lambda: mol.mol_paged_attention(q, c, c, table, at, workspace=moved(cuda(4096, dtype=torch.uint8)),
                                        stream=side),
    ]
    for i, call in enumerate(wrong):
        with pytest.raises(ValueError, match="current device"):
            call()
            pytest.fail(f"call {i} was taken")
    assert not binding.calls


def test_what_is_handed_over(binding):  # noqa: F811
    """Strides of operands and caches; one token, head or page has none that matters."""
    rows = cuda(5, 8, 64)
    at = cuda(5, dtype=i32)
    kc = cuda(3, 2, 8, 64).transpose(1, 2)  # [pages, page, heads, D] of pages laid out heads first
    side = Stream(0x20)
    mol.mol_cache_append(rows[:, 4:6], rows[:, 6:], kc, kc, at, stream=side)
    name, a = binding.calls[-1]
    assert name == "mol_cache_append" and a[1:3] == (512, 64) and a[4:6] == (512, 64)
    c = a[10]
    assert (c.page_stride, c.token_stride, c.head_stride) == (2 * 8 * 64, 64, 8 * 64)
    assert (c.num_pages, c.page_size, c.num_heads, c.head_dim) == (3, 8, 2, 64)
    one = cuda(1, 1, 64).as_strided((1, 1, 64), (7, 3, 1))  # strides that no call could take
    mol.mol_rope(one, at[:1].clone(), mol.Rope(cuda(32, dtype=f32)), stream=side)
    assert binding.calls[-1][1][1] % 8 == 0 and binding.calls[-1][1][2] % 8 == 0
    with pytest.raises(ValueError, match="same strides"):
        mol.mol_cache_append(rows[:, 4:6], rows[:, 6:], kc, cuda(3, 8, 2, 64), at, stream=side)
