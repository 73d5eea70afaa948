"""GPU tests of the MoE block's operators against the float64 oracle.

Bounds, derived before the first run. A bf16 output carries one rounding, at most 2^-9 of its
value; 2^-8 leaves the same again for fp32 arithmetic around it. A product accumulated in fp32
adds at most 2^-16 of the sum of its terms' magnitudes (K * 2^-24 at K = 256, and rounding errors
of either sign beyond). mol_moe_forward reads its activations rounded to bf16: 2^-8 of the
magnitudes behind each output more. Router weights: a quotient of fp32 exponentials and a sum of at
most 1024 of them, 1e-5. Ids are exact.
"""

import math

import numpy as np
import pytest

from oracle import block_oracle as bo
from tests.gpu_util import mol_lib, torch_cuda

pytestmark = pytest.mark.gpu

ROUND, ACC = 2.0 ** -8, 2.0 ** -16
FORMATS = [0, 32, 64, 128]


@pytest.fixture(scope="module")
def env():
    return torch_cuda(), mol_lib()


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, want, bound, what):
    got = f64(got)
    assert got.shape == want.shape
    err = np.abs(got - want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {np.argwhere(bad)[:4].tolist()} off by {err[bad][:4]}"


def randn(torch, g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def strided(torch, t, pad=8, fill=float("nan")):
    """The same rows on the GPU inside a wider buffer of `fill`."""
    wide = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    wide[:, :t.shape[1]] = t.cuda()
    return wide[:, :t.shape[1]]


# ------------------------------------------------------------------------------------------ norm
@pytest.mark.parametrize("H", [8, 16, 120, 256, 264, 1000, 1024, 2048, 2056, 4096, 4104, 8192, 8200,
                               16384])
@pytest.mark.parametrize("T,post,gate,layout", [
    (1, True, "row", "plain"), (5, False, "none", "strided"), (3, True, "token", "strided"),
    (130, True, "none", "inplace"), (7, False, "token", "plain")])
def test_norm(env, H, T, post, gate, layout):
    torch, mol = env
    g = torch.Generator().manual_seed(H * 7 + T)
    y, r = randn(torch, g, T, H, std=3.0), randn(torch, g, T, H, std=2.0)
    y[T // 2] = 0
    pre, pw = randn(torch, g, H) + 1, randn(torch, g, H) + 1
    gt = {"none": None, "row": randn(torch, g, H), "token": randn(torch, g, T, H)}[gate]
    dy, dr = (strided(torch, y), strided(torch, r, 16)) if layout == "strided" else (y.cuda(), r.cuda())
    kw = {}
    if layout == "inplace":
        kw = dict(residual_out=dr, normed=dy)
    elif layout == "strided":
        kw = dict(residual_out=strided(torch, torch.zeros(T, H, dtype=torch.bfloat16), 24, 7.0),
                  normed=strided(torch, torch.zeros(T, H, dtype=torch.bfloat16), 8, 7.0))
    ro, n = mol.mol_block_norm(dy, dr, pre.cuda(), post_weight=pw.cuda() if post else None,
                               gate=None if gt is None else gt.cuda(), residual_scale=-0.75,
                               eps=1e-5, **kw)
    want = bo.block_norm(f64(y), f64(r), f64(pre), f64(pw) if post else None,
                         None if gt is None else f64(gt), -0.75, 1e-5)
    scale = np.sqrt((want[0] ** 2).mean())
    # residual + s * n: the sum may cancel, so its terms' fp32 errors count beside the rounding
    terms = np.abs(f64(r)) + np.abs(want[0] - f64(r))
    close(ro, want[0], ROUND * np.abs(want[0]) + 2.0 ** -20 * terms, "residual_out")
    close(n, want[1], ROUND * np.abs(want[1]) + 2.0 ** -18 * np.abs(f64(pre)) * terms / scale,
          "normed")
    if layout == "strided":
        for t, pad in ((ro, 24), (n, 8)):
            wide = t.as_strided((T, H + pad), (H + pad, 1))
            assert torch.all(wide[:, H:] == 7.0)


def test_norm_without_the_second_norm_and_with_bad_rows(env):
    """No pre_weight: no second output. A row of NaN or infinity stays its own."""
    torch, mol = env
    g = torch.Generator().manual_seed(3)
    y, r, w = randn(torch, g, 4, 256), randn(torch, g, 4, 256), randn(torch, g, 256)
    y[1, 7], y[2, 9] = float("nan"), float("inf")
    ro, n = mol.mol_block_norm(y.cuda(), r.cuda(), None, post_weight=w.cuda())
    assert n is None
    ok = [0, 3]
    want, _ = bo.block_norm(f64(y)[ok], f64(r)[ok], None, f64(w))
    close(ro[ok], want, ROUND * np.abs(want) + 1e-5, "residual_out")
    assert torch.isnan(ro[1]).all()
    assert mol.mol_block_norm(y[:0].cuda(), r[:0].cuda(), w.cuda())[1].shape == (0, 256)


# ----------------------------------------------------------------------------------------- router
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,E,k,renorm,scale", [
    (1, 1, 1, True, 1.0), (3, 8, 2, False, 2.5), (5, 31, 8, True, 1.0), (6, 33, 32, False, 1.0),
    (9, 128, 8, True, 1.0), (4, 200, 6, False, 0.5), (7, 256, 8, True, 2.0), (3, 500, 10, False, 1.0),
    (2, 1024, 32, True, 1.0), (517, 64, 4, True, 1.0)])
def test_route(env, dtype, T, E, k, renorm, scale):
    torch, mol = env
    g = torch.Generator().manual_seed(T * E + k)
    v = torch.randn(T, E, generator=g) * 3
    if dtype == "bf16" or E % 2:
        v = v.to(torch.bfloat16)     # many ties
    v = v.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    v = v.masked_fill(torch.rand(T, E, generator=g) < 0.3, -math.inf)
    v[0] = 0.0                       # all equal: ids 0, 1, ...
    if T > 2:
        v[1] = -math.inf             # nothing to take
        v[2] = torch.finfo(v.dtype).min
        v[2, E // 2] = 1.0
    if T > 5:
        v[3, ::2] = math.nan
        v[4, E // 3] = math.inf
        v[5, ::2], v[5, 1::2] = -0.0, 0.0
    wide = torch.full((T, E + 3), math.inf, dtype=v.dtype, device="cuda")
    wide[:, :E] = v.cuda()
    ids, w = mol.mol_moe_route(wide[:, :E], k, renormalize=renorm, scale=scale)
    want_ids, want_w = bo.moe_route(f64(v), k, renorm, scale)
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    close(w, want_w, 1e-5 * np.abs(want_w) + 1e-37, "weights")
    assert bool((w[ids < 0] == 0).all())


# ---------------------------------------------------------------------------------------- experts
def make_weights(torch, mol, g, lead, K, group):
    """(device weights, their float64 values [*lead, K])."""
    if group == 0:
        w = randn(torch, g, *lead, K, std=K ** -0.5)
        return w.cuda(), f64(w)
    q = torch.randint(0, 16, (*lead, K), generator=g)
    s = (torch.rand(*lead, -(-K // group), generator=g) + 0.5) * (0.2 * K ** -0.5)
    w = mol.w4_pack(q, s, group)
    # what padding holds must not matter
    used = -(-K // group)
    w.scales[..., used:] = float("nan")
    flat = w.qweight.view(-1, w.qweight.shape[-1])
    vals = bo.w4_values(flat.numpy(), f64(w.scales).reshape(flat.shape[0], -1), K, group)
    return mol.W4(w.qweight.cuda(), w.scales.cuda(), K, group), vals.reshape(*lead, K)


def make_ids(torch, g, T, E, k, kind):
    ids = torch.stack([torch.randperm(max(E, k), generator=g)[:k] % E for _ in range(T)])
    if kind == "hot":
        ids[:, 0] = E - 1
        for j in range(1, k):
            ids[:, j] = ids[:, j] % max(E - 1, 1)
    elif kind == "dropped":
        ids[torch.rand(T, k, generator=g) < 0.4] = -1
        ids[T // 2] = -1
    elif kind == "none":
        ids[:] = -1
    elif kind == "repeated":
        ids[:] = torch.randint(0, E, (T, 1), generator=g)
    elif kind == "outside":
        ids[::2, 0], ids[1::2, -1] = E, -7
        ids[0, -1] = 2 ** 31 - 1
    return ids.to(torch.int32)


# T, E, k, H, I, ids
SHAPES = [
    (1, 8, 2, 256, 128, "plain"), (1, 1, 1, 8, 8, "plain"), (2, 3, 2, 16, 24, "plain"),
    (7, 4, 2, 40, 136, "plain"), (8, 40, 8, 128, 64, "dropped"), (9, 5, 3, 264, 72, "repeated"),
    (17, 16, 4, 1000, 200, "plain"), (23, 128, 8, 256, 48, "plain"), (33, 8, 2, 136, 768, "outside"),
    (64, 6, 3, 520, 104, "hot"), (65, 4, 4, 72, 88, "hot"), (128, 16, 8, 256, 40, "plain"),
    (128, 2, 2, 64, 64, "repeated"), (12, 8, 2, 2048, 32, "none"), (3, 300, 8, 128, 16, "plain"),
    (1, 1024, 16, 64, 32, "plain"), (31, 24, 32, 64, 16, "plain"), (128, 8, 8, 1288, 8, "hot"),
    (2, 3, 2, 10248, 16, "plain"), (40, 3, 2, 4104, 520, "plain"), (100, 2, 1, 2600, 1032, "plain"),
    (1, 2, 1, 32, 20000, "plain"), (64, 12, 4, 6152, 40, "dropped")]


def run_experts(env, shape, group, delta, seed=0):
    torch, mol = env
    T, E, k, H, I, kind = shape
    g = torch.Generator().manual_seed(seed + T * 131 + E * 17 + H + I + group)
    x, ids = randn(torch, g, T, H), make_ids(torch, g, T, E, k, kind)
    weights = torch.rand(T, k, generator=g) * 2 - 0.5
    gu, gu64 = make_weights(torch, mol, g, (E, 2 * I), H, group)
    dn, dn64 = make_weights(torch, mol, g, (E, H), I, group)
    dgu, ddn = (randn(torch, g, T * k, 2 * I), randn(torch, g, T * k, H)) if delta else (None, None)
    ids_np, w_np = ids.numpy(), f64(weights)
    dx = strided(torch, x) if delta else x.cuda()
    act = torch.full((T * k, I), 7.0, dtype=torch.bfloat16, device="cuda")
    mol.mol_moe_gate_up(dx, ids.cuda(), gu, act=act,
                        delta=None if dgu is None else strided(torch, dgu))
    want, slack = bo.moe_gate_up(f64(x), ids_np, gu64, None if dgu is None else f64(dgu))
    valid = ~np.isnan(want[:, 0])
    close(act[torch.from_numpy(valid).cuda()], want[valid],
          ROUND * np.abs(want[valid]) + ACC * slack[valid], "act")
    assert bool((act[torch.from_numpy(~valid).cuda()] == 7.0).all()), "row of an absent pair written"
    # the second half on activations of its own; absent pairs' rows hold NaN
    a = randn(torch, g, T * k, I)
    a[torch.from_numpy(~valid)] = float("nan")
    out = strided(torch, torch.full((T, H), 5.0, dtype=torch.bfloat16), 8, 3.0)
    mol.mol_moe_down(a.cuda(), ids.cuda(), weights.cuda(), dn, out=out,
                     delta=None if ddn is None else strided(torch, ddn))
    want_out, mag = bo.moe_down(f64(a), ids_np, w_np, dn64, None if ddn is None else f64(ddn))
    close(out, want_out, ROUND * np.abs(want_out) + ACC * mag, "out")
    assert bool((out.as_strided((T, H + 8), (H + 8, 1))[:, H:] == 3.0).all())
    if not delta:
        both = mol.mol_moe_forward(dx, ids.cuda(), weights.cuda(), gu, dn)
        want_both, mag = bo.moe_down(want, ids_np, w_np, dn64)
        # bf16 activations (ROUND of each) carry the first product's accumulation error too
        slack_out = bo.moe_down(np.nan_to_num(slack), ids_np, np.abs(w_np), np.abs(dn64))[0]
        close(both, want_both, ROUND * np.abs(want_both) + (ROUND + ACC) * mag + ACC * slack_out,
              "forward")


@pytest.mark.parametrize("group", FORMATS)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_experts(env, shape, group):
    run_experts(env, shape, group, delta=False)


@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("shape", SHAPES[3:11], ids=lambda s: "-".join(map(str, s)))
def test_experts_with_deltas(env, shape, group):
    run_experts(env, shape, group, delta=True)


@pytest.mark.parametrize("group", [0, 128])
def test_experts_weights_that_no_token_takes_are_not_read_into_results(env, group):
    """Experts without a token hold NaN; one token of NaN leaves the others as they are."""
    torch, mol = env
    g = torch.Generator().manual_seed(5)
    T, E, k, H, I = 9, 12, 2, 256, 64
    x = randn(torch, g, T, H)
    ids = torch.randint(0, 6, (T, 1), generator=g) * 2
    ids = torch.cat([ids, (ids + 2) % 12], 1).to(torch.int32)
    weights = torch.rand(T, k, generator=g).cuda()
    gu, _ = make_weights(torch, mol, g, (E, 2 * I), H, group)
    dn, _ = make_weights(torch, mol, g, (E, H), I, group)
    clean = mol.mol_moe_forward(x.cuda(), ids.cuda(), weights, gu, dn)
    for w in (gu, dn):
        (w.scales if group else w)[1::2] = float("nan")
    x[4] = float("nan")
    got = mol.mol_moe_forward(x.cuda(), ids.cuda(), weights, gu, dn)
    rest = [t for t in range(T) if t != 4]
    assert torch.equal(got[rest], clean[rest]) and torch.isnan(got[4]).all()


@pytest.mark.parametrize("group", [0, 32])
def test_experts_are_bit_reproducible_and_follow_the_stream(env, group):
    torch, mol = env
    g = torch.Generator().manual_seed(6)
    T, E, k, H, I = 40, 24, 6, 512, 128
    gu, _ = make_weights(torch, mol, g, (E, 2 * I), H, group)
    dn, _ = make_weights(torch, mol, g, (E, H), I, group)
    ids = make_ids(torch, g, T, E, k, "plain").cuda()
    weights = torch.rand(T, k, generator=g).cuda()
    xs = [randn(torch, g, T, H).cuda() for _ in range(3)]
    want = [mol.mol_moe_forward(x, ids, weights, gu, dn) for x in xs]
    for _ in range(5):
        for x, w in zip(xs, want):
            assert torch.equal(mol.mol_moe_forward(x, ids, weights, gu, dn), w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x = xs[0] * 1.0
        got = mol.mol_moe_forward(x, ids, weights, gu, dn)
    side.synchronize()
    assert torch.equal(got, want[0])
    # a captured call replays on new contents of its buffers
    x, out = xs[0].clone(), torch.empty_like(want[0])
    act = torch.empty(T * k, I, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        mol.mol_moe_forward(x, ids, weights, gu, dn, out=out, act=act)
    for i in (1, 2):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])


def test_experts_launch_two_kernels(env):
    torch, mol = env
    g = torch.Generator().manual_seed(7)
    gu, _ = make_weights(torch, mol, g, (4, 64), 64, 0)
    dn, _ = make_weights(torch, mol, g, (4, 64), 32, 0)
    ids = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    w = torch.ones(3, 1, device="cuda")
    before = mol.mol_launch_count()
    mol.mol_moe_forward(randn(torch, g, 3, 64).cuda(), ids, w, gu, dn)
    assert mol.mol_launch_count() - before == 2


@pytest.mark.parametrize("group", [0, 128])
def test_experts_past_32_bit_offsets(env, group):
    """The last of enough experts that its weights lie past 2^32 bytes (and elements)."""
    torch, mol = env
    H, I = 4096, 2048
    E = (2 ** 32 // (2 * I * H) if group == 0 else 2 ** 33 // (2 * I * H)) + 2
    g = torch.Generator().manual_seed(8)
    gu1, gu64 = make_weights(torch, mol, g, (1, 2 * I), H, group)
    dn1, dn64 = make_weights(torch, mol, g, (1, H), I, group)

    def among(w1):
        if group == 0:
            w = torch.empty((E, *w1.shape[1:]), dtype=w1.dtype, device="cuda")
            w[-1:] = w1
            return w
        q = torch.empty((E, *w1.qweight.shape[1:]), dtype=torch.uint8, device="cuda")
        s = torch.empty((E, *w1.scales.shape[1:]), dtype=torch.bfloat16, device="cuda")
        q[-1:], s[-1:] = w1.qweight, w1.scales
        return mol.W4(q, s, w1.in_features, group)

    x = randn(torch, g, 2, H)
    ids = torch.tensor([[E - 1], [E - 1]], dtype=torch.int32)
    weights = torch.tensor([[1.0], [0.5]])
    got = mol.mol_moe_forward(x.cuda(), ids.cuda(), weights.cuda(), among(gu1), among(dn1))
    act, slack = bo.moe_gate_up(f64(x), np.zeros((2, 1), int), gu64)
    want, mag = bo.moe_down(act, np.zeros((2, 1), int), f64(weights), dn64)
    slack_out = bo.moe_down(slack, np.zeros((2, 1), int), f64(weights), np.abs(dn64))[0]
    close(got, want, ROUND * np.abs(want) + (ROUND + ACC) * mag + ACC * slack_out, "forward")


# ----------------------------------------------------------------------------------------- linear
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,K,N", [
    (1, 8, 1), (1, 256, 17), (2, 128, 64), (3, 1000, 33), (7, 2048, 40), (8, 264, 300), (9, 96, 2049),
    (16, 520, 7), (17, 1024, 129), (33, 640, 65), (64, 136, 150), (64, 2056, 16), (1, 5000, 5),
    (5, 256, 40000), (20, 64, 9001)])
def test_linear(env, T, K, N, group):
    torch, mol = env
    g = torch.Generator().manual_seed(T + K * 3 + N)
    x = randn(torch, g, T, K)
    if N <= 4096:
        w, w64 = make_weights(torch, mol, g, (N,), K, group)
    else:  # the oracle's nibble loop is slow there: the packing is checked above
        w, _ = make_weights(torch, mol, g, (1,), K, group)
        q = torch.randint(0, 256, (N, w.qweight.shape[1]), dtype=torch.uint8, generator=g)
        s = (torch.rand(N, w.scales.shape[1], generator=g) * 0.01).to(torch.bfloat16)
        w64 = f64(mol.w4_unpack(mol.W4(q, s, K, group)))
        w = mol.W4(q.cuda(), s.cuda(), K, group)
    out = strided(torch, torch.full((T, N), 5.0, dtype=torch.bfloat16), 3, 2.0)
    got = mol.mol_w4_linear(strided(torch, x), w, out=out)
    want, mag = f64(x) @ w64.T, np.abs(f64(x)) @ np.abs(w64).T
    close(got, want, ROUND * np.abs(want) + ACC * mag, "out")
    assert bool((out.as_strided((T, N + 3), (N + 3, 1))[:, N:] == 2.0).all())
    assert torch.equal(mol.mol_w4_linear(x.cuda(), w), got)


# --------------------------------------------------------------------------------------- refusals
def test_binding_refusals(env):
    torch, mol = env
    bf, dev = torch.bfloat16, "cuda"
    x, ids = torch.zeros(2, 64, dtype=bf, device=dev), torch.zeros(2, 1, dtype=torch.int32, device=dev)
    w = torch.ones(2, 1, device=dev)
    gu, dn = torch.zeros(4, 32, 64, dtype=bf, device=dev), torch.zeros(4, 64, 16, dtype=bf, device=dev)
    mol.mol_moe_forward(x, ids, w, gu, dn)
    for bad in [(x.float(), ids, w, gu, dn), (x, ids.long(), w, gu, dn), (x, ids, w.double(), gu, dn),
                (x.cpu(), ids, w, gu, dn)]:
        with pytest.raises(TypeError):
            mol.mol_moe_forward(*bad)
    for bad in [(x, ids, w, gu[..., :32], dn), (x, ids, w, gu, dn[..., :8]), (x, ids, w[:1], gu, dn),
                (x, ids, w, gu, dn[:3]), (x, ids, w, gu.transpose(1, 2), dn),
                (x, ids, w, mol.W4(gu, gu, 64, 48), dn)]:
        with pytest.raises(ValueError):
            mol.mol_moe_forward(*bad)
    with pytest.raises(mol.MolError):   # more tokens than the call takes
        mol.mol_moe_forward(x.repeat(65, 1), ids.repeat(65, 1), w.repeat(65, 1), gu, dn)
    with pytest.raises(mol.MolError):
        mol.mol_moe_route(torch.zeros(2, 4, device=dev), 5)
    with pytest.raises(ValueError):
        mol.mol_block_norm(x, x[:, :32], None)
    with pytest.raises(TypeError):
        mol.mol_w4_linear(x, gu)
    with pytest.raises(ValueError):
        mol.mol_moe_gate_up(x, ids, gu, delta=torch.zeros(2, 16, dtype=bf, device=dev))


# ---------------------------------------------------------------------------------- checked build
@pytest.mark.parametrize("group", FORMATS)
def test_checked_build_records_nothing(env, group):
    """The checked build runs the same shapes: every index stays in its buffer."""
    torch, mol = env
    from moe_lora_virtual_gb300.build import build_library

    with mol.use_library(build_library(checked=True)):
        mol.mol_take_check_record()
        for shape in SHAPES:
            run_experts(env, shape, group, delta=False, seed=1)
        if group:
            for T, K, N in ((1, 256, 17), (16, 520, 700), (64, 136, 150), (5, 256, 9000)):
                test_linear(env, T, K, N, group)
        rec = mol.mol_take_check_record()
        assert rec.count == 0, f"{rec.count} failed checks, first {rec.site_name} value {rec.value}"
        assert mol.mol_take_fault_flags() == 0


# ---------------------------------------------------------------------------------- bounded waits
@pytest.mark.parametrize("group", [0, 64])
def test_wait_runs_out_sets_flag_then_device_recovers(env, group):
    """With the producer warps issuing nothing every wait gives up: the calls return, bit 0 is
    reported, no activation was written; the same call right after is right, with no bit set."""
    torch, mol = env
    g = torch.Generator().manual_seed(11)
    T, E, k, H, I = 9, 8, 2, 512, 128
    x, ids = randn(torch, g, T, H).cuda(), make_ids(torch, g, T, E, k, "plain").cuda()
    weights = torch.rand(T, k, generator=g).cuda()
    gu, _ = make_weights(torch, mol, g, (E, 2 * I), H, group)
    dn, _ = make_weights(torch, mol, g, (E, H), I, group)
    want = mol.mol_moe_forward(x, ids, weights, gu, dn)
    assert mol.mol_take_fault_flags() == 0
    act = torch.full((T * k, I), 7.0, dtype=torch.bfloat16, device="cuda")
    try:
        mol.mol_debug_wait_test(True, 2_000_000)  # waits give up after 2 ms
        mol.mol_moe_forward(x, ids, weights, gu, dn, act=act)
        flags = mol.mol_take_fault_flags()
    finally:
        mol.mol_debug_wait_test(False, 0)
    assert flags == 1 and bool((act == 7.0).all())
    assert torch.equal(mol.mol_moe_forward(x, ids, weights, gu, dn), want)
    assert mol.mol_take_fault_flags() == 0


@pytest.mark.parametrize("delta", [False, True])
@pytest.mark.parametrize("group", FORMATS)
@pytest.mark.parametrize("shape", [
    (17, 4, 2, 200, 72, "plain"), (64, 6, 3, 520, 104, "hot"), (128, 3, 8, 264, 40, "dropped"),
    (40, 5, 4, 2056, 264, "repeated"), (65, 1, 1, 72, 1032, "plain"), (33, 7, 2, 8, 8, "outside")],
    ids=lambda s: "-".join(map(str, s)))
def test_down_in_both_forms(env, shape, group, delta):
    """The second half in one kernel and, with a workspace, as fp32 products and their sums."""
    torch, mol = env
    T, E, k, H, I, kind = shape
    g = torch.Generator().manual_seed(11 + T + H + group)
    ids, w = make_ids(torch, g, T, E, k, kind), torch.rand(T, k, generator=g) * 2 - 0.5
    a = randn(torch, g, T * k, I)
    a[(ids.flatten() < 0) | (ids.flatten() >= E)] = float("nan")
    dn, dn64 = make_weights(torch, mol, g, (E, H), I, group)
    d = randn(torch, g, T * k, H) if delta else None
    want, mag = bo.moe_down(f64(a), ids.numpy(), f64(w), dn64, None if d is None else f64(d))
    a, ids, w, d = a.cuda(), ids.cuda(), w.cuda(), None if d is None else d.cuda()
    data, scales = (dn.qweight, dn.scales) if group else (dn, None)
    out = torch.full((T, H), 5.0, dtype=torch.bfloat16, device="cuda")
    args = [a.data_ptr(), ids.data_ptr(), w.data_ptr(), T, k, E, H, I, data.data_ptr(),
            None if scales is None else scales.data_ptr(), group,
            None if d is None else d.data_ptr(), 0 if d is None else H]
    assert mol.library().mol_moe_down(*args, out.data_ptr(), H, None) == 0
    close(out, want, ROUND * np.abs(want) + ACC * mag, "one kernel")
    need = mol.mol_moe_workspace_bytes(T, k, E, H, I, group)
    ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")  # (fp32 NaN)
    before = mol.mol_launch_count()
    got = mol.mol_moe_down(a, ids, w, dn, delta=d, workspace=ws)
    assert mol.mol_launch_count() - before == (2 if need else 1)
    close(got, want, ROUND * np.abs(want) + ACC * mag, "with a workspace")
    if need:
        with pytest.raises(mol.MolError):
            mol.mol_moe_down(a, ids, w, dn, delta=d, workspace=ws[:-4])
        with pytest.raises(TypeError):
            mol.mol_moe_down(a, ids, w, dn, delta=d, workspace=ws.cpu())


@pytest.mark.parametrize("group", [0, 64])
def test_example_model_step(env, group):
    """A step of the example model: a graph's replay equals the calls, and the logits those of the
    same step in float64 with bf16 rounding where the model holds bf16. Each such rounding is at
    most ROUND / 2 of its value; a layer has fewer than ten in a row and the norms keep magnitudes
    near one, so 2 layers and the head stay below 32 roundings, taken in the mean square."""
    import importlib.util
    import os
    torch, mol = env
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "decode_layers.py")
    spec = importlib.util.spec_from_file_location("decode_layers", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    T, k, E, L = 13, 4, 32, 4
    model = example.Model(tokens=T, group=group, seed=3)
    g = torch.Generator().manual_seed(4)
    tokens = torch.randint(0, 5000, (T,), generator=g).cuda()
    lora = torch.randint(-1, L, (T,), generator=g).to(torch.int32).cuda()
    got = model(tokens, lora)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = model(tokens, lora)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, got)

    def dense(w):
        return mol.w4_unpack(w).double() if isinstance(w, mol.W4) else w.double()

    def rms(v, w):
        return (v * w.double() * torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-6))

    residual, y = model.embed[tokens].double(), 0.0
    for lay in model.layers:
        residual = (residual + y).bfloat16().double()
        x = rms(residual, lay.norm).bfloat16().double()
        # the choice is the device's: it is exact for its own logits, and ties within a rounding
        ids, w = mol.mol_moe_route(x.bfloat16() @ lay.router.T, k)
        gu, dn = dense(lay.gate_up), dense(lay.down)
        y = torch.zeros_like(x)
        for t in range(T):
            for j in range(k):
                e, l = int(ids[t, j]), int(lora[t])
                h, v = gu[e] @ x[t], e + l * E
                if l >= 0:
                    r = lay.b_gu.shape[-1]
                    a = (lay.a_gu[v].double() @ x[t]).view(2, r)
                    h = h + lay.scale * torch.cat([lay.b_gu[v, s * (len(h) // 2):][:len(h) // 2].double() @ a[s]
                                                   for s in range(2)])
                gate, up = h.chunk(2)
                act = (gate * torch.sigmoid(gate) * up).bfloat16().double()
                o = dn[e] @ act
                if l >= 0:
                    o = o + lay.scale * (lay.b_dn[v].double() @ (lay.a_dn[v].double() @ act))
                y[t] += w[t, j].double() * o
        y = y.bfloat16().double()
    residual = (residual + y).bfloat16().double()
    want = rms(residual, model.norm).bfloat16().double() @ dense(model.head).T
    err = ((got.double() - want).square().mean() / want.square().mean()).sqrt().item()
    assert err < 32 ** 0.5 * ROUND / 2, err


@pytest.mark.parametrize("group", [0, 64])
def test_native_calls_equal_the_python_path(env, group, monkeypatch):
    torch, mol = env
    from moe_lora_virtual_gb300 import block
    assert block._native is not None, "the native calls are not built"
    g = torch.Generator().manual_seed(9)
    T, E, k, H, I = 21, 6, 2, 264, 72
    x, r, gate, w = (randn(torch, g, *s).cuda() for s in ((T, H), (T, H), (T, H), (H,)))
    gu, _ = make_weights(torch, mol, g, (E, 2 * I), H, group)
    dn, _ = make_weights(torch, mol, g, (E, H), I, group)
    head, _ = make_weights(torch, mol, g, (40,), H, group or 32)
    d = randn(torch, g, T * k, 2 * I).cuda(), randn(torch, g, T * k, H).cuda()
    logits = torch.randn(T, E, generator=g).cuda()
    taken = []
    real = block._native

    class Count:
        def __getattr__(self, name):
            def call(*a):
                out = getattr(real, name)(*a)
                taken.append(out is not None)
                return out
            return call

    def everything(x, r):
        out = [*mol.mol_block_norm(x, r, w, post_weight=w, gate=gate, residual_scale=0.5, eps=1e-5),
               mol.mol_block_norm(x, r, None, gate=w)[0]]
        ids, tw = mol.mol_moe_route(logits, k, renormalize=False, scale=2.0)
        act = mol.mol_moe_gate_up(x, ids, gu)
        return out + [ids, tw, act, mol.mol_moe_gate_up(x, ids, gu, delta=d[0]),
                      mol.mol_moe_down(act, ids, tw, dn), mol.mol_moe_down(act, ids, tw, dn, delta=d[1]),
                      mol.mol_moe_forward(x, ids, tw, gu, dn), mol.mol_w4_linear(x, head),
                      *mol.mol_moe_route(logits.to(torch.bfloat16), 1)]

    monkeypatch.setattr(block, "_native", Count())
    got = everything(x, r)
    assert len(taken) == 10 and all(taken)
    taken.clear()
    wide = everything(strided(torch, x.cpu()), r)  # rows with a stride
    assert all(taken)
    monkeypatch.setattr(block, "_native", None)
    for a, b, c in zip(got, wide, everything(x, r)):
        assert a.dtype == b.dtype == c.dtype and torch.equal(a, c) and torch.equal(b, c)
    monkeypatch.setattr(block, "_native", real)
    with pytest.raises(ValueError):
        mol.mol_moe_forward(x, torch.zeros(T, k, dtype=torch.int32, device="cuda"),
                            torch.zeros(T, k + 1, device="cuda"), gu, dn)
    with pytest.raises(mol.MolError):
        mol.mol_moe_route(logits, E + 1)


@pytest.mark.parametrize("H", [8, 256, 264, 512, 520])
def test_norm_of_many_short_rows(env, H):
    """2051 rows: several a block, the last block's not all there."""
    torch, mol = env
    g = torch.Generator().manual_seed(H)
    T = 2051
    y, r, gate = randn(torch, g, T, H, std=3.0), randn(torch, g, T, H), randn(torch, g, T, H)
    w = 1 + randn(torch, g, H, std=0.2)
    ro, n = mol.mol_block_norm(strided(torch, y), strided(torch, r), w.cuda(), post_weight=w.cuda(),
                               gate=gate.cuda(), residual_scale=0.5)
    want, want_n = bo.block_norm(f64(y), f64(r), f64(w), f64(w), f64(gate), 0.5)
    # one rounding each, and the fp32 sums' error as in the tests above
    close(ro, want, ROUND * np.abs(want) + ACC, "residual")
    close(n, want_n, ROUND * np.abs(want_n) + ACC, "normed")
