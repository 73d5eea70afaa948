"""CPU checks of the MoE block's entry points: exports, refusals, the 4-bit layout, the oracle.

Refusals: no call here reaches a kernel, the arguments are rejected first.
"""

import ctypes
import os
import re

import numpy as np
import pytest

from oracle import block_oracle as bo
from tests.test_abi_cpu import mol, needs_nvcc  # noqa: F401  (fixture)

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
INVALID, UNSUPPORTED = -1, -3


def header():
    return open(os.path.join(ROOT, "include", "mol_block.h")).read()


@needs_nvcc
def test_exports_every_declared_symbol(mol):
    src = re.sub(r"/\*.*?\*/", "", header(), flags=re.S)
    names = set(re.findall(r"\b(mol_\w+)\s*\(", src))
    assert names == set(mol.BLOCK_EXPORTS) == set(mol.BLOCK_SIGS)
    for path in (mol.LIB_PATH, mol.CHECKED_LIB_PATH):
        with mol.use_library(path) as lib:
            for n in names:
                assert hasattr(lib, n), n
                declared = re.search(r"\b%s\s*\((.*?)\);" % n, src, flags=re.S).group(1)
                assert len(declared.split(",")) == len(mol.BLOCK_SIGS[n][1]), n


def test_limits_match_header():
    from moe_lora_virtual_gb300 import block

    for name, value in re.findall(r"#define (MOL_\w+) (\d+)", header()):
        assert getattr(block, name) == int(value), name


def norm_args(**kw):
    a = dict(y=P(16), ys=64, r=P(16), rs=64, post=P(16), gate=P(16), gs=0, scale=1.0, pre=P(16),
             eps=1e-6, T=3, H=64, ro=P(16), ros=64, n=P(16), ns=64)
    a.update(kw)
    return [*a.values(), None]


@needs_nvcc
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=-8), INVALID), (dict(H=60), UNSUPPORTED),
    (dict(H=16392), UNSUPPORTED), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(eps=float("inf")), INVALID), (dict(y=None), INVALID), (dict(r=None), INVALID),
    (dict(ro=None), INVALID), (dict(n=None), INVALID), (dict(pre=None), INVALID),
    (dict(ys=56), INVALID), (dict(ys=68), UNSUPPORTED), (dict(ns=56), INVALID),
    (dict(gs=32), INVALID), (dict(gs=68), UNSUPPORTED), (dict(gate=P(20)), UNSUPPORTED),
    (dict(post=P(18)), UNSUPPORTED), (dict(y=P(24)), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED)])
def test_norm_refusals(mol, kw, status):
    assert mol.library().mol_block_norm(*norm_args(**kw)) == status


@needs_nvcc
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=9), INVALID),
    (dict(dt=2), INVALID), (dict(stride=7), INVALID), (dict(renorm=2), INVALID),
    (dict(E=1025, stride=2000), UNSUPPORTED), (dict(E=64, stride=64, k=33), UNSUPPORTED),
    (dict(T=(1 << 22) + 1), UNSUPPORTED), (dict(x=None), INVALID), (dict(x=P(18)), UNSUPPORTED),
    (dict(x=P(17), dt=1), UNSUPPORTED), (dict(ids=None), INVALID), (dict(w=None), INVALID)])
def test_route_refusals(mol, kw, status):
    a = dict(x=P(16), dt=0, stride=8, T=3, E=8, k=2, renorm=1, scale=1.0, ids=P(16), w=P(16))
    a.update(kw)
    assert mol.library().mol_moe_route(*a.values(), None) == status


SHAPE_REFUSALS = [
    (dict(T=-1), INVALID), (dict(k=0), INVALID), (dict(E=0), INVALID), (dict(H=0), INVALID),
    (dict(I=0), INVALID), (dict(T=129, k=1), UNSUPPORTED), (dict(T=128, k=9), UNSUPPORTED),
    (dict(E=1025), UNSUPPORTED), (dict(H=60), UNSUPPORTED), (dict(I=60), UNSUPPORTED),
    (dict(H=65544), UNSUPPORTED), (dict(I=65544), UNSUPPORTED), (dict(ids=None), INVALID)]
WEIGHT_REFUSALS = [
    (dict(w=None), INVALID), (dict(w=P(24)), UNSUPPORTED), (dict(G=48), UNSUPPORTED),
    (dict(G=256), UNSUPPORTED), (dict(G=-32), UNSUPPORTED), (dict(G=0), INVALID),
    (dict(s=None), INVALID), (dict(s=P(20)), UNSUPPORTED)]


@needs_nvcc
@pytest.mark.parametrize("kw,status", SHAPE_REFUSALS + WEIGHT_REFUSALS + [
    (dict(x=None), INVALID), (dict(xs=56), INVALID), (dict(xs=68), UNSUPPORTED),
    (dict(x=P(20)), UNSUPPORTED), (dict(act=None), INVALID), (dict(act=P(18)), UNSUPPORTED),
    (dict(ds=120), INVALID), (dict(ds=132), UNSUPPORTED), (dict(d=P(20)), UNSUPPORTED)])
def test_gate_up_refusals(mol, kw, status):
    a = dict(x=P(16), xs=64, ids=P(16), T=2, k=2, E=4, H=64, I=64, w=P(16), s=P(16), G=32, d=P(16),
             ds=128, act=P(16))
    a.update(kw)
    if "H" in kw and kw["H"] > 64:
        a["xs"] = kw["H"]
    assert mol.library().mol_moe_gate_up(*a.values(), None) == status


@needs_nvcc
@pytest.mark.parametrize("kw,status", SHAPE_REFUSALS + WEIGHT_REFUSALS + [
    (dict(tw=None), INVALID), (dict(act=None), INVALID), (dict(out=None), INVALID),
    (dict(os=56), INVALID), (dict(os=68), UNSUPPORTED), (dict(out=P(18)), UNSUPPORTED),
    (dict(ds=56), INVALID), (dict(d=P(20)), UNSUPPORTED)])
def test_down_refusals(mol, kw, status):
    a = dict(act=P(16), ids=P(16), tw=P(16), T=2, k=2, E=4, H=64, I=64, w=P(16), s=P(16), G=32,
             d=P(16), ds=64, out=P(16), os=64)
    a.update(kw)
    assert mol.library().mol_moe_down(*a.values(), None) == status


@needs_nvcc
@pytest.mark.parametrize("kw,status", SHAPE_REFUSALS + WEIGHT_REFUSALS + [
    (dict(w2=None), INVALID), (dict(s2=None), INVALID), (dict(w2=P(20)), UNSUPPORTED),
    (dict(act=None), INVALID), (dict(out=None), INVALID), (dict(os=56), INVALID)])
def test_forward_refusals(mol, kw, status):
    a = dict(x=P(16), xs=64, ids=P(16), tw=P(16), T=2, k=2, E=4, H=64, I=64, w=P(16), s=P(16),
             w2=P(16), s2=P(16), G=32, act=P(16), out=P(16), os=64)
    a.update(kw)
    if "H" in kw and kw["H"] > 64:
        a["xs"] = kw["H"]
    assert mol.library().mol_moe_forward(*a.values(), None) == status


@needs_nvcc
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(K=0), INVALID), (dict(N=0), INVALID), (dict(T=65), UNSUPPORTED),
    (dict(K=60), UNSUPPORTED), (dict(K=65544, xs=65544), UNSUPPORTED), (dict(xs=56), INVALID),
    (dict(xs=68), UNSUPPORTED), (dict(os=6), INVALID), (dict(out=None), INVALID),
    (dict(out=P(17)), UNSUPPORTED), (dict(G=0, s=None), UNSUPPORTED), (dict(G=16), UNSUPPORTED),
    (dict(s=None), INVALID), (dict(w=None), INVALID), (dict(x=None), INVALID)])
def test_linear_refusals(mol, kw, status):
    a = dict(x=P(16), xs=64, T=2, K=64, N=7, w=P(16), s=P(16), G=32, out=P(16), os=7)
    a.update(kw)
    assert mol.library().mol_w4_linear(*a.values(), None) == status


@needs_nvcc
def test_no_tokens_is_ok_without_a_device(mol):
    lib = mol.library()
    assert lib.mol_block_norm(*norm_args(T=0, y=None, ro=None)) == 0
    assert lib.mol_moe_route(None, 0, 8, 0, 8, 2, 1, 1.0, None, None, None) == 0
    assert lib.mol_moe_forward(None, 64, None, None, 0, 2, 4, 64, 64, None, None, None, None, 0,
                               None, None, 64, None) == 0
    assert lib.mol_w4_linear(None, 64, 0, 64, 7, None, None, 32, None, 7, None) == 0


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("K", [8, 40, 128, 256, 328, 640])
def test_pack_layout_against_the_oracle(group, K):
    from moe_lora_virtual_gb300 import w4_pack, w4_unpack

    g = torch.Generator().manual_seed(K + group)
    q = torch.randint(0, 16, (5, K), generator=g)
    s = torch.rand(5, -(-K // group), generator=g) + 0.1
    w = w4_pack(q, s, group)
    Kp = -(-K // 256) * 256
    assert w.qweight.shape == (5, Kp // 2) and w.scales.shape == (5, Kp // group)
    sb = s.to(torch.bfloat16).double().numpy()
    want = (q.numpy() - 8.0) * np.repeat(sb, group, 1)[:, :K]
    got = bo.w4_values(w.qweight.numpy(), w.scales.double().numpy(), K, group)
    assert np.array_equal(got, want)
    assert np.array_equal(w4_unpack(w).double().numpy(), want)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantize_is_within_half_a_step(group):
    from moe_lora_virtual_gb300 import w4_quantize, w4_unpack

    g = torch.Generator().manual_seed(group)
    w = torch.randn(6, 200, generator=g)
    w[3] = 0
    p = w4_quantize(w, group)
    groups = -(-200 // group)
    step = p.scales[:, :groups].float().repeat_interleave(group, 1)[:, :200]
    # half a step; the largest magnitude may be clipped by what rounding its scale to bf16 took off
    assert torch.all((w4_unpack(p) - w).abs() <= step * 0.5 + w.abs() * 2 ** -8 + 1e-7)
    assert torch.all(w4_unpack(p)[3] == 0)


def test_pack_refusals():
    from moe_lora_virtual_gb300 import w4_pack, w4_quantize

    q = torch.zeros(2, 64, dtype=torch.int64)
    with pytest.raises(ValueError):
        w4_pack(q, torch.ones(2, 4), 16)
    with pytest.raises(ValueError):
        w4_pack(q, torch.ones(2, 3), 32)
    with pytest.raises(ValueError):
        w4_pack(q + 16, torch.ones(2, 2), 32)
    with pytest.raises(ValueError):
        w4_quantize(torch.zeros(2, 64), 48)


def test_oracle_route_hand_worked():
    inf = np.inf
    logits = np.array([[1.0, 3.0, 3.0, 2.0], [-inf, -inf, 0.0, -inf], [-inf] * 4,
                       [np.nan, 5.0, -inf, inf]])
    ids, w = bo.moe_route(logits, 2, True, 1.0)
    assert ids.tolist() == [[1, 2], [2, -1], [-1, -1], [3, 1]]
    assert np.allclose(w, [[0.5, 0.5], [1.0, 0.0], [0.0, 0.0], [1.0, 0.0]])
    _, w = bo.moe_route(logits[:1], 2, False, 2.0)
    assert np.allclose(w, 2 / (2 + np.exp(-2) + np.exp(-1)))


def test_oracle_experts_hand_worked():
    x = np.array([[1.0, 2.0]])
    gu = np.array([[[1.0, 0.0], [0.0, 1.0]], [[0.0, 1.0], [1.0, 1.0]]])   # I = 1
    dn = np.array([[[1.0], [2.0]], [[-1.0], [0.5]]])
    ids = np.array([[1, -1]])
    act, _ = bo.moe_gate_up(x, ids, gu)
    assert np.isclose(act[0, 0], 2 / (1 + np.exp(-2)) * 3) and np.isnan(act[1, 0])
    out, _ = bo.moe_down(np.nan_to_num(act), ids, np.array([[0.5, 9.0]]), dn)
    assert np.allclose(out, 0.5 * act[0, 0] * dn[1][:, 0])


def test_oracle_norm_hand_worked():
    y, r = np.array([[3.0, 4.0]]), np.array([[1.0, 1.0]])
    ro, n = bo.block_norm(y, r, np.array([1.0, 2.0]), post=np.array([1.0, 1.0]),
                          gate=np.array([2.0, 0.0]), scale=0.5, eps=0.0)
    m = np.sqrt(12.5)
    assert np.allclose(ro, [[1 + 3 / m, 1.0]])
    q = np.sqrt(((1 + 3 / m) ** 2 + 1) / 2)
    assert np.allclose(n, [[(1 + 3 / m) / q, 2 / q]])


@needs_nvcc
@pytest.mark.parametrize("kw,status", [
    (dict(ws=None), -2), (dict(wsb=40 * 64 * 4 - 1), -2), (dict(ws=P(20)), UNSUPPORTED),
    (dict(tw=None), INVALID), (dict(act=None), INVALID), (dict(T=129), UNSUPPORTED)])
def test_split_refusals(mol, kw, status):
    """40 pairs of 4-bit experts take the workspace of one fp32 row for each."""
    assert mol.mol_moe_workspace_bytes(20, 2, 4, 64, 64, 32) == 40 * 64 * 4
    a = dict(act=P(16), ids=P(16), tw=P(16), T=20, k=2, E=4, H=64, I=64, w=P(16), s=P(16), G=32,
             d=None, ds=0, ws=P(16), wsb=40 * 64 * 4, out=P(16), os=64)
    a.update(kw)
    assert mol.library().mol_moe_down_split(*a.values(), None) == status
    f = dict(x=P(16), xs=64, ids=P(16), tw=P(16), T=20, k=2, E=4, H=64, I=64, w=P(16), s=P(16),
             w2=P(16), s2=P(16), G=32, act=P(16), ws=P(16), wsb=40 * 64 * 4, out=P(16), os=64)
    f.update(kw)
    assert mol.library().mol_moe_forward_split(*f.values(), None) == status


@needs_nvcc
def test_workspace_sizes(mol):
    """Few pairs, and bf16 experts of few tokens, need none; nor do sizes that are refused."""
    for shape in [(0, 8, 16, 64, 64, 32), (4, 8, 16, 64, 64, 32), (40, 8, 128, 64, 64, 0),
                  (129, 1, 4, 64, 64, 32), (20, 2, 4, 60, 64, 32)]:
        assert mol.mol_moe_workspace_bytes(*shape) == 0, shape
    assert mol.mol_moe_workspace_bytes(40, 8, 16, 64, 64, 0) == 320 * 64 * 4


@needs_nvcc
def test_native_calls_leave_everything_unusual_to_the_python_path(mol):
    """Wrong kinds, counts, types, devices: None, and no exception is left behind."""
    native = pytest.importorskip("moe_lora_virtual_gb300._block_native")
    import torch
    x, w = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(3, 8, 64, dtype=torch.bfloat16)
    ids = torch.zeros(2, 1, dtype=torch.int32)
    f = ctypes.cast(mol.library().mol_block_norm, ctypes.c_void_p).value
    for name, args in [("block_norm", (f, x, x, None, None, None, 1.0, 1e-6)),
                       ("moe_route", (f, x, 1, 1, 1.0)),
                       ("moe_gate_up", (f, x, ids, w, None, 64, 0, None)),
                       ("moe_down", (f, f, x, ids, x, w, None, 64, 0, None)),
                       ("moe_forward", (f, f, x, ids, x, w, None, 64, 0, w, None, 64, 0)),
                       ("w4_linear", (f, x, x, x, 64, 32))]:
        call = getattr(native, name)
        for bad in [args, args[:-1], (), (0, *args[1:]), (None, *args[1:]), (f, None, *args[2:]),
                    (f, "x", *args[2:]), (2 ** 80, *args[1:]), tuple([x] * len(args)),
                    (*args[:-1], 2 ** 70), (*args[:-1], "x")]:
            assert call(*bad) is None, (name, bad)
