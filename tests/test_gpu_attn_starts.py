"""GPU tests of paged attention whose q_starts decrease, which no batch has: nothing is written, in out or past
the scratch, and no wait runs out; starts past the rows that do not decrease once they are taken as the nearer
end are taken so."""

import pytest

from tests import attn_util as au
from tests.gpu_util import mol_lib, torch_cuda
from tests.test_gpu_attn import attend

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


def shuffled(torch, p, starts):
    return dict(p, starts=torch.tensor(starts, dtype=torch.int32))


# Few rows (16 and 32 a block), many (tensor copies, gathered tokens), 256 values a head; undivided and in parts
@pytest.mark.parametrize("kv", [100, 4000])
@pytest.mark.parametrize("n,D,page", [
    (1, 64, 16), (1, 128, 16), (1, 256, 16), (3, 64, 16), (60, 64, 16), (200, 64, 16), (60, 64, 5), (60, 128, 16),
    (200, 128, 5), (90, 256, 16)])
def test_starts_that_decrease(build, n, D, page, kv):
    torch, mol = build
    p = au.problem(torch, D + n, [(n, kv), (n, kv // 2), (n, kv // 3), (n, 1 + kv // 9)], 8, 2, D, page, lead=1)
    T = 1 + 4 * n
    want = attend(build, p)
    ws = torch.full((mol.mol_paged_attention_workspace_bytes(4, T, 8, 2, D) + (1 << 20),), 0x5A, dtype=torch.uint8,
                    device="cuda")
    for starts in ([0, n, T, 2 * n, T], [T, 0, T, 0, T], [0, T, 0, T, T - 1], [3, 2, 2, 2, 2], [1 << 30, 0, 1, 1, 1],
                   [0, 1, 1, 1, -1]):
        got = attend(build, shuffled(torch, p, starts), fill=7.0, workspace=ws[:-(1 << 20)])
        assert bool((got == 7.0).all()), starts
        assert bool((ws[-(1 << 20):] == 0x5A).all())
    assert mol.mol_take_fault_flags() == 0
    assert torch.equal(attend(build, p), want)


@pytest.mark.parametrize("B", [130, 400])
def test_one_start_of_many_decreases(build, B):
    """More sequences than threads: wherever the one lies. The last one is set past the rows: taken as their
    end, 2 B, it does not decrease, and the sequence before it has its rows too."""
    torch, mol = build
    p = au.problem(torch, B, [(2, 9)] * B, 4, 2, 64, 16)
    for at in (1, 127, 128, B - 1):
        starts = list(range(0, 2 * B + 1, 2))
        starts[at] = starts[at + 1] + 1
        got = attend(build, shuffled(torch, p, starts), fill=7.0)
        if at == B - 1:
            near = [min(x, 2 * B) for x in starts]
            assert near == sorted(near)
            assert torch.equal(got, attend(build, shuffled(torch, p, near), fill=7.0))
        else:
            assert bool((got == 7.0).all()), at


def test_parts_that_would_pass_the_last_thread_block(build):
    """Starts whose sequences would be cut into more tiles than were dealt out: 152 thread blocks' list went on
    to a 153rd."""
    torch, mol = build
    lens, starts = [29399, 54888, 30000, 30000, 42], [3192, 2484, 324, 2875, 2815, 4094]
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(5249, 2, 256, generator=g, device="cuda").to(torch.bfloat16)
    kc = torch.randn(700, 128, 1, 256, generator=g, device="cuda").to(torch.bfloat16)
    table = torch.randint(700, (5, 8192), generator=g, device="cuda").to(torch.int32)
    out = torch.full_like(q, 7.0)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    mol.mol_paged_attention(q, kc, kc, table, i32(lens), i32(starts), out=out)
    assert bool((out == 7.0).all()) and mol.mol_take_fault_flags() == 0


def test_starts_that_decrease_past_the_ends_are_the_ends(build):
    torch, mol = build
    p = au.problem(torch, 3, [(40, 60), (3, 48)], 4, 2, 64, 16)
    want = attend(build, p)
    assert torch.equal(attend(build, shuffled(torch, p, [-3, 40, 43])), want)
    for starts in ([-1, -9, 43], [0, 1 << 30, 50]):  # (0, 0, 43 and 0, 43, 43)
        near = [min(max(x, 0), 43) for x in starts]
        assert torch.equal(attend(build, shuffled(torch, p, starts), fill=7.0),
                           attend(build, shuffled(torch, p, near), fill=7.0))
