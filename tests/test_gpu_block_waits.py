"""GPU tests of the bounded waits in the calls of the MoE block that the two-kernel layer does not
reach: the 4-bit linear (short and long rows, one team and many) and the split form."""

import pytest

from tests import test_gpu_block as tb
from tests.test_gpu_block import env  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def stalled(mol, call):
    """Fault bits of a call whose token warps issue nothing; its waits give up after 2 ms."""
    assert mol.mol_take_fault_flags() == 0
    try:
        mol.mol_debug_wait_test(True, 2_000_000)
        call()
        return mol.mol_take_fault_flags()
    finally:
        mol.mol_debug_wait_test(False, 0)


@pytest.mark.parametrize("T,K,N", [(1, 2048, 512), (16, 4096, 700), (40, 256, 9000)])
def test_linear(env, T, K, N):
    torch, mol = env
    g = torch.Generator().manual_seed(K)
    x = tb.randn(torch, g, T, K).cuda()
    w = mol.w4_quantize(torch.randn(N, K, generator=g).cuda(), 64)
    want = mol.mol_w4_linear(x, w)
    out = torch.full_like(want, 7.0)
    assert stalled(mol, lambda: mol.mol_w4_linear(x, w, out=out)) == 1
    assert bool((out == 7.0).all())
    assert torch.equal(mol.mol_w4_linear(x, w), want) and mol.mol_take_fault_flags() == 0


@pytest.mark.parametrize("group", [0, 32])
def test_split_form(env, group):
    torch, mol = env
    g = torch.Generator().manual_seed(12)
    T, E, k, H, I = 40, 8, 2, 512, 128
    x, ids = tb.randn(torch, g, T, H).cuda(), tb.make_ids(torch, g, T, E, k, "plain").cuda()
    w = torch.rand(T, k, generator=g).cuda()
    gu, _ = tb.make_weights(torch, mol, g, (E, 2 * I), H, group)
    dn, _ = tb.make_weights(torch, mol, g, (E, H), I, group)
    need = mol.mol_moe_workspace_bytes(T, k, E, H, I, group)
    assert need
    want = mol.mol_moe_forward(x, ids, w, gu, dn)
    act = torch.full((T * k, I), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    out = torch.full_like(want, 7.0)
    assert stalled(mol, lambda: mol.mol_moe_forward(x, ids, w, gu, dn, out=out, act=act,
                                                    workspace=ws)) == 1
    assert bool((act == 7.0).all()) and bool((ws == 0).all())
    assert bool((out == 0).all())  # the sums of the untouched workspace
    assert torch.equal(mol.mol_moe_forward(x, ids, w, gu, dn), want)
    assert mol.mol_take_fault_flags() == 0
