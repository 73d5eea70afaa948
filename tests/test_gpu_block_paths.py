"""GPU tests of every way in which the experts and the 4-bit linear deal out their work: whole rows and
pieces of them, one and two token slots, short rings, teams of one warp and of several, one, two and
four token tiles, clusters of 1, 2 and 4 blocks. test_block_plan_cpu.py checks that the shapes below
reach all of them. Plain form and bounds in float64 on the device; the bounds are those of
test_gpu_block.py (a contraction of 20000 inputs is 1250 accumulations, each off by at most 2^-23 of a
partial sum, which stays below a 50th of the sum of magnitudes: 2^-18 of it)."""

import pytest

from tests.test_gpu_block import ACC, ROUND, env  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

# group, tokens, slots, experts, hidden, inter
EXPERTS = [
    # gate_up: rings of two chunks, pieces of rows, several warps a team
    (32, 62, 2, 35, 4968, 520), (0, 5, 1, 1, 6320, 8), (128, 8, 1, 1, 8560, 8),
    (0, 113, 3, 4, 2800, 12488), (32, 48, 15, 50, 2096, 128), (0, 34, 1, 1, 2928, 8),
    (0, 6, 1, 1, 17536, 8), (32, 6, 1, 1, 18392, 8), (32, 18, 36, 130, 9968, 280),
    (128, 62, 9, 10, 4824, 1168), (0, 46, 1, 1, 8040, 8), (32, 110, 2, 2, 4632, 8),
    (0, 15, 2, 2, 336, 8), (64, 13, 1, 1, 1784, 8), (128, 2, 1, 2, 1096, 8), (0, 2, 1, 1, 136, 8),
    # the split form, the same
    (32, 21, 15, 64, 488, 4776), (0, 28, 2, 8, 8, 5768), (128, 36, 1, 5, 8, 6176),
    (0, 36, 17, 35, 2776, 2912), (128, 68, 14, 113, 104, 2464), (0, 123, 2, 2, 8, 2848),
    (64, 119, 1, 1, 8, 2336), (64, 26, 12, 46, 424, 2592), (128, 19, 2, 6, 8, 4544),
    (64, 21, 2, 6, 8, 12496), (32, 80, 1, 6, 3320, 4896), (0, 18, 2, 2, 8, 4512),
    (128, 47, 1, 1, 8, 5704), (64, 38, 1, 6, 8, 1056), (0, 40, 2, 3, 64, 8200),
    (64, 64, 4, 4, 200, 6152), (0, 36, 2, 2, 8, 280), (0, 36, 1, 5, 8, 280),
    (0, 21, 2, 6, 8, 2952), (0, 93, 1, 1, 8, 296), (0, 8, 5, 5, 16, 12592), (32, 112, 1, 1, 8, 8),
    # down in one kernel: clusters, pieces of rows
    (0, 1, 2, 2, 8, 3920), (64, 4, 2, 2, 24, 5528), (0, 98, 2, 2, 16, 408), (64, 124, 2, 2, 8, 296),
    (0, 30, 6, 25, 8, 120), (0, 107, 3, 3, 8, 200), (32, 7, 1, 1, 8, 6072), (0, 7, 1, 1, 8, 2808),
    (128, 107, 1, 1, 8, 1912), (0, 10, 1, 1, 8, 1632)]
# group, tokens, inputs, outputs
LINEAR = [
    (32, 49, 5264, 5117), (32, 8, 4496, 1), (32, 46, 2752, 4479), (32, 30, 2064, 1),
    (64, 31, 1528, 11400), (128, 19, 3600, 9762), (128, 19, 8, 9737), (64, 20, 64, 10001),
    (32, 32, 2056, 10001), (128, 64, 8200, 300), (64, 7, 12248, 98900), (64, 8, 9664, 17),
    (32, 12, 9576, 38547), (64, 16, 20000, 3001), (128, 20, 9640, 33), (128, 29, 10304, 25577),
    (64, 20, 9576, 10340), (32, 27, 20000, 10001)]


def random_weights(torch, mol, g, lead, K, group):
    if group == 0:
        w = torch.empty(*lead, K, dtype=torch.bfloat16, device="cuda")
        for rows in w.view(-1, K).split(1 << 16):
            rows.copy_(torch.randn(rows.shape, generator=g, device="cuda") * K ** -0.5)
        return w
    Kp, used = -(-K // 256) * 256, -(-K // group)
    q = torch.randint(0, 256, (*lead, Kp // 2), dtype=torch.uint8, generator=g, device="cuda")
    s = (torch.rand(*lead, Kp // group, generator=g, device="cuda") + 0.5) * (0.2 * K ** -0.5)
    s[..., used:] = float("nan")  # what padding holds must not matter
    return mol.W4(q, s.to(torch.bfloat16), K, group)


def rows64(mol, w, *at):
    if isinstance(w, mol.W4):
        return mol.w4_unpack(w._replace(qweight=w.qweight[at], scales=w.scales[at])).double()
    return w[at].double()


def near(torch, got, want, bound, what):
    bad = ~((got.double() - want).abs() <= bound)
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()}, first at {bad.nonzero()[0].tolist()}"


def run_experts(torch, mol, group, T, k, E, H, I):
    g = torch.Generator(device="cuda").manual_seed(T + H + I)
    x = torch.randn(T, H, generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.rand(T, E, generator=g, device="cuda").argsort(1)[:, :k].to(torch.int32).contiguous()
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, -1, ids)
    ids[0, 0] = E - 1
    w = torch.rand(T, k, generator=g, device="cuda") * 2 - 0.5
    gu, dn = (random_weights(torch, mol, g, lead, K, group)
              for lead, K in (((E, 2 * I), H), ((E, H), I)))
    act = torch.full((T * k, I), 7.0, dtype=torch.bfloat16, device="cuda")
    mol.mol_moe_gate_up(x, ids, gu, act=act)
    a = torch.randn(T * k, I, generator=g, device="cuda").to(torch.bfloat16)
    a[ids.view(-1) < 0] = float("nan")
    one = torch.full((T, H), 7.0, dtype=torch.bfloat16, device="cuda")
    data, scales = (dn.qweight, dn.scales) if group else (dn, None)
    assert mol.library().mol_moe_down(
        a.data_ptr(), ids.data_ptr(), w.data_ptr(), T, k, E, H, I, data.data_ptr(),
        None if scales is None else scales.data_ptr(), group, None, 0, one.data_ptr(), H,
        torch.cuda.current_stream().cuda_stream) == 0
    need = mol.mol_moe_workspace_bytes(T, k, E, H, I, group)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda") if need else None  # (NaN)
    split = mol.mol_moe_down(a, ids, w, dn, workspace=ws)

    assert bool((act[ids.view(-1) < 0] == 7.0).all())
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for e in sorted(set(ids.view(-1).tolist()) - {-1}):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        pairs = t * k + j
        v, m = (f(x[t].double()) @ f(rows64(mol, gu, e)).T for f in (lambda z: z, torch.abs))
        gate, up = v[:, :I], v[:, I:]
        silu = gate * torch.sigmoid(gate)
        near(torch, act[pairs], silu * up,
             ROUND * (silu * up).abs() + ACC * (1.1 * m[:, :I] * up.abs() + silu.abs() * m[:, I:]), "act")
        rows, scale = rows64(mol, dn, e), w[t, j].double().unsqueeze(1)
        want.index_add_(0, t, scale * (a[pairs].double() @ rows.T))
        mag.index_add_(0, t, scale.abs() * (a[pairs].double().abs() @ rows.abs().T))
    bound = ROUND * want.abs() + ACC * mag
    near(torch, one, want, bound, "one kernel")
    near(torch, split, want, bound, "split form" if need else "binding")


def run_linear(torch, mol, group, T, K, N):
    g = torch.Generator(device="cuda").manual_seed(T + K + N)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    w = random_weights(torch, mol, g, (N,), K, group)
    wide = torch.full((T, N + 5), 2.0, dtype=torch.bfloat16, device="cuda")
    got = mol.mol_w4_linear(x, w, out=wide[:, :N])
    step = max(1, (1 << 27) // K)
    for n in range(0, N, step):
        rows = rows64(mol, w, slice(n, n + step))
        want, mag = x.double() @ rows.T, x.double().abs() @ rows.abs().T
        near(torch, got[:, n:n + step], want, ROUND * want.abs() + ACC * mag, f"outputs from {n} on")
    assert bool((wide[:, N:] == 2.0).all())


@pytest.fixture(params=["checked", "release"])
def build(request, env):
    """Both builds; in the checked one every index stays in its buffer. No wait runs out."""
    torch, mol = env
    from moe_lora_virtual_gb300.build import build_library

    with mol.use_library(build_library(checked=request.param == "checked")):
        mol.mol_take_check_record()
        mol.mol_take_fault_flags()
        yield torch, mol
        rec = mol.mol_take_check_record()
        assert rec.count == 0, f"{rec.count} failed checks, first {rec.site_name} value {rec.value}"
        assert mol.mol_take_fault_flags() == 0


@pytest.mark.parametrize("shape", EXPERTS, ids=lambda s: "-".join(map(str, s)))
def test_experts(build, shape):
    run_experts(*build, *shape)


@pytest.mark.parametrize("shape", LINEAR, ids=lambda s: "-".join(map(str, s)))
def test_linear(build, shape):
    run_linear(*build, *shape)


def test_linear_an_entry_a_launch(env):
    """So many outputs that the entries' rows pass 2^30 together: a launch for each 16 tokens. The
    first and last outputs are looked at; the weights between them are whatever memory holds."""
    torch, mol = env
    T, K, group = 33, 8, 128
    N = (1 << 30) // 3 + 777
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 100 GB of free device memory")
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    w = mol.W4(torch.empty(N, 128, dtype=torch.uint8, device="cuda"),
               torch.empty(N, 2, dtype=torch.bfloat16, device="cuda"), K, group)
    ends = [slice(0, 40), slice(N // 2, N // 2 + 40), slice(N - 40, N)]
    for s in ends:
        part = random_weights(torch, mol, g, (40,), K, group)
        w.qweight[s], w.scales[s] = part.qweight, part.scales
    before = mol.mol_launch_count()
    got = mol.mol_w4_linear(x, w)
    assert mol.mol_launch_count() - before == 3
    for s in ends:
        rows = rows64(mol, w, s)
        want, mag = x.double() @ rows.T, x.double().abs() @ rows.abs().T
        near(torch, got[:, s], want, ROUND * want.abs() + ACC * mag, "ends")
