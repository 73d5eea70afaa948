"""GPU tests of the MoE block's calls with `stream=`: what they allocate outlives its kernels."""

import pytest

from tests import test_gpu_block as tb
from tests.test_gpu_block import env  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("group", [0, 64])
def test_scratch_is_not_handed_out_while_the_stream_is_busy(env, group, handle):
    """The calls wait behind 20 ms of other work of their stream. Meanwhile the current stream
    allocates tensors of the sizes of their scratch and outputs and fills them."""
    torch, mol = env
    g = torch.Generator().manual_seed(21)
    T, E, k, H, I = 60, 8, 4, 512, 128
    gu, _ = tb.make_weights(torch, mol, g, (E, 2 * I), H, group)
    dn, _ = tb.make_weights(torch, mol, g, (E, H), I, group)
    ids = tb.make_ids(torch, g, T, E, k, "plain").cuda()
    w = torch.rand(T, k, generator=g).cuda()
    x, norm_w = tb.randn(torch, g, T, H).cuda(), tb.randn(torch, g, H).cuda()
    need = mol.mol_moe_workspace_bytes(T, k, E, H, I, group)
    assert need, "the case is to take a workspace"

    def step(**kw):
        _, n = mol.mol_block_norm(x, x, norm_w, **kw)
        act = mol.mol_moe_gate_up(n, ids, gu, **kw)
        return mol.mol_moe_forward(n, ids, w, gu, dn, **kw), mol.mol_moe_down(act, ids, w, dn, **kw)

    want = step()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(40_000_000)
        got = step(stream=side.cuda_stream if handle else side)
        junk = []
        for _ in range(8):
            junk.append(torch.full((T * k, I), float("nan"), dtype=torch.bfloat16, device="cuda"))
            junk.append(torch.full((T, H), float("nan"), dtype=torch.bfloat16, device="cuda"))
            junk.append(torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(bool(torch.isnan(j).all()) if j.dtype == torch.bfloat16 else bool((j == 255).all())
                   for j in junk)
