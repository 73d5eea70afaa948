"""CPU checks of the attention half's entry points: exports, refusals, frequencies, the oracle.

Refusals: no call here reaches a kernel, the arguments are rejected first.
"""

import ctypes
import math
import os
import re

import numpy as np
import pytest

from oracle import attn_oracle as ao
from tests.test_abi_cpu import mol, needs_nvcc  # noqa: F401  (fixture)

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
OK, INVALID, CAPACITY, UNSUPPORTED = 0, -1, -2, -3
INF, NAN = float("inf"), float("nan")


def header():
    return open(os.path.join(ROOT, "include", "mol_attn.h")).read()


@needs_nvcc
def test_exports_every_declared_symbol(mol):
    src = re.sub(r"/\*.*?\*/", "", header(), flags=re.S)
    names = set(re.findall(r"\b(mol_\w+)\s*\(", src))
    assert names == set(mol.ATTN_EXPORTS) == set(mol.ATTN_SIGS)
    for path in (mol.LIB_PATH, mol.CHECKED_LIB_PATH):
        with mol.use_library(path) as lib:
            for n in names:
                assert hasattr(lib, n), n
                declared = re.search(r"\b%s\s*\((.*?)\);" % n, src, flags=re.S).group(1)
                assert len(declared.split(",")) == len(mol.ATTN_SIGS[n][1]), n


def test_limits_match_header():
    from moe_lora_virtual_gb300 import attention

    for name, value in re.findall(r"#define (MOL_\w+) (\d+)", header()):
        assert getattr(attention, name) == int(value), name


def test_structures_match_header():
    from moe_lora_virtual_gb300 import attention

    for struct, fields in (("mol_rope_table", attention._RopeTable), ("mol_paged_cache", attention._PagedCache)):
        body = re.search(r"typedef struct %s \{(.*?)\}" % struct, header(), flags=re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        names = []
        for line in body.split(";"):
            names += [re.sub(r".*[\s*]", "", n.strip()) for n in line.split(",") if n.strip()]
        assert names == [n for n, _ in fields._fields_]


def table(freq=P(16), R=32, inter=0, m=1.0):
    from moe_lora_virtual_gb300.attention import _RopeTable

    return _RopeTable(freq, R, inter, m)


def cache(**kw):
    from moe_lora_virtual_gb300.attention import _PagedCache

    a = dict(k=P(16), v=P(16), ps=2 * 8 * 64, ts=2 * 64, hs=64, pages=4, size=8, heads=2, D=64)
    a.update(kw)
    return _PagedCache(*a.values())


ROPE_TABLE = [
    (dict(freq=None), INVALID), (dict(R=0), INVALID), (dict(R=-16), INVALID), (dict(R=80), INVALID),
    (dict(R=24), UNSUPPORTED), (dict(R=2), UNSUPPORTED), (dict(m=INF), INVALID), (dict(m=NAN), INVALID),
    (dict(inter=2), INVALID), (dict(inter=-1), INVALID)]


@needs_nvcc
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(D=0), INVALID), (dict(D=60), UNSUPPORTED),
    (dict(D=520), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED), (dict(H=65537), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(out=None), INVALID), (dict(pos=None), INVALID), (dict(rope=None), INVALID),
    (dict(xt=56), INVALID), (dict(xh=56), INVALID), (dict(xt=260), UNSUPPORTED), (dict(oh=68), UNSUPPORTED),
    (dict(x=P(24)), UNSUPPORTED), (dict(out=P(18)), UNSUPPORTED), (dict(T=0), OK),
    *[(dict(rope=r), s) for r, s in ROPE_TABLE]])
def test_rope_refusals(mol, kw, status):
    a = dict(x=P(16), xt=256, xh=64, pos=P(16), rope={}, T=3, H=4, D=64, out=P(16), ot=256, oh=64)
    a.update(kw)
    a["rope"] = None if a["rope"] is None else table(**a["rope"])
    assert mol.library().mol_rope(*a.values(), None) == status


CACHE = [
    (dict(pages=-1), INVALID), (dict(size=0), INVALID), (dict(heads=0), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(ps=56), INVALID), (dict(ts=56), INVALID), (dict(hs=56), INVALID),
    (dict(ps=1028), UNSUPPORTED), (dict(ts=132), UNSUPPORTED), (dict(hs=68), UNSUPPORTED),
    (dict(k=P(8)), UNSUPPORTED), (dict(v=P(20)), UNSUPPORTED), (dict(pages=1 << 28), UNSUPPORTED),
    (dict(pages=1 << 40, size=1 << 30), UNSUPPORTED)]


@needs_nvcc
@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INVALID), (dict(T=1 << 31), UNSUPPORTED), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(slots=None), INVALID), (dict(pos=None), INVALID), (dict(kt=56), INVALID), (dict(vh=68), UNSUPPORTED),
    (dict(q=None), INVALID), (dict(qo=None), INVALID), (dict(rope=None), INVALID), (dict(Hq=0), INVALID),
    (dict(qt=56), INVALID), (dict(qoh=60), INVALID), (dict(T=0), OK),
    (dict(cache=dict(D=60)), UNSUPPORTED), (dict(cache=dict(D=16)), INVALID),  # (turned 32)
    *[(dict(rope=r), s) for r, s in ROPE_TABLE], *[(dict(cache=c), s) for c, s in CACHE]])
def test_append_refusals(mol, kw, status):
    a = dict(k=P(16), kt=128, kh=64, v=P(16), vt=128, vh=64, slots=P(16), pos=P(16), rope={}, T=3, cache={},
             q=P(16), qt=256, qh=64, Hq=4, qo=P(16), qot=256, qoh=64)
    a.update(kw)
    a["rope"] = None if a["rope"] is None else table(**a["rope"])
    a["cache"] = cache(**a["cache"])
    assert mol.library().mol_cache_append(*a.values(), None) == status


@needs_nvcc
@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(T=-1), INVALID), (dict(H=0), INVALID), (dict(H=3), INVALID),
    (dict(H=2 * 65), UNSUPPORTED), (dict(mp=-1), INVALID), (dict(win=-1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID), (dict(scale=3e38), INVALID),
    (dict(starts=None), INVALID), (dict(st=3), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(qt=56), INVALID), (dict(oh=68), UNSUPPORTED),
    (dict(q=P(8)), UNSUPPORTED), (dict(mp=1 << 28, st=1 << 28), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED),
    (dict(mp=(1 << 28) - 64, st=1 << 28), UNSUPPORTED),  # (a tile's end past 2^31)
    (dict(T=1 << 29), UNSUPPORTED), (dict(B=1 << 24), UNSUPPORTED), (dict(ws=None), CAPACITY),
    (dict(wsb=64), CAPACITY), (dict(ws=P(8)), UNSUPPORTED), (dict(T=0), OK), (dict(B=0), OK),
    (dict(cache=dict(D=96, hs=96, ts=192, ps=1536)), UNSUPPORTED), (dict(cache=dict(D=32)), UNSUPPORTED),
    *[(dict(cache=c), s) for c, s in CACHE]])
def test_attention_refusals(mol, kw, status):
    a = dict(q=P(16), qt=256, qh=64, cache={}, table=P(16), st=4, mp=4, lens=P(16), starts=P(16), B=2, T=3, H=4,
             scale=0.125, win=0, out=P(16), ot=256, oh=64, ws=P(256), wsb=1 << 40)
    a.update(kw)
    a["cache"] = cache(**a["cache"])
    assert mol.library().mol_paged_attention(*a.values(), None) == status


@needs_nvcc
def test_workspace_sizes(mol):
    size = mol.mol_paged_attention_workspace_bytes
    assert size(0, 0, 4, 2, 64) == 0 and size(1, 1, 4, 3, 64) == 0 and size(1, 1, 4, 2, 96) == 0
    for D in (64, 128, 256):
        assert 0 < size(4, 9, 8, 2, D) < 128 << 20


@needs_nvcc
def test_native_calls_leave_everything_unusual_to_the_python_path(mol):
    """Wrong kinds, counts, types, devices: None, and no exception is left behind."""
    native = pytest.importorskip("moe_lora_virtual_gb300._block_native")
    x, c = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 8, 2, 64, dtype=torch.bfloat16)
    i, f = torch.zeros(2, dtype=torch.int32), torch.zeros(32)
    e = ctypes.cast(mol.library().mol_rope, ctypes.c_void_p).value
    for name, args in [("rope", (e, x, i, f, 0, 1.0)),
                       ("cache_append", (e, x, x, c, c, i, i, f, 0, 1.0, x)),
                       ("paged_attention", (e, e, x, c, c, i.view(2, 1), i, None, 0.1, 0))]:
        call = getattr(native, name)
        for bad in [args, args[:-1], (), (0, *args[1:]), (None, *args[1:]), (e, None, *args[2:]),
                    (e, "x", *args[2:]), (2 ** 80, *args[1:]), tuple([x] * len(args)),
                    (*args[:-1], 2 ** 70), (*args[:-1], "x")]:
            assert call(*bad) is None, (name, bad)


# ----------------------------------------------------------------------------------- frequencies
def test_frequencies(mol):
    f = mol.rope_frequencies
    assert f(8, 10000.0).inv_freq.tolist() == pytest.approx([1, 0.1, 0.01, 0.001], rel=1e-6)
    assert f(8, scaling="linear", factor=4.0).inv_freq.tolist() == pytest.approx(
        [0.25, 0.025, 0.0025, 0.00025], rel=1e-6)
    a, b = f(64).inv_freq, f(64, scaling="base", factor=8.0).inv_freq
    assert float(b[0]) == 1.0 and float(b[-1]) == pytest.approx(float(a[-1]) / 8, rel=1e-6)
    r = f(64, scaling="parts", factor=4.0, trained=4096, interleaved=True)
    turns = 4096 * a.double() / (2 * math.pi)
    assert r.interleaved and r.magnitude == pytest.approx(0.1 * math.log(4) + 1)
    ratio = (a / r.inv_freq).double()
    assert torch.all(ratio[turns >= 34] == 1) and torch.all((ratio[turns < 0.7] - 4).abs() < 1e-5)
    assert torch.all(ratio[1:] >= ratio[:-1] - 1e-6)
    assert f(64, scaling="parts", factor=4.0, trained=4096, magnitude=1.0).magnitude == 1.0


@pytest.mark.parametrize("args,kw", [
    ((7,), {}), ((0,), {}), ((8,), dict(scaling="other")), ((8,), dict(factor=0.5)), ((8, 1.0), {}),
    ((8,), dict(scaling="parts", factor=2.0)), ((8,), dict(scaling="parts", factor=2.0, trained=9, slow_turns=3,
                                                             fast_turns=2))])
def test_frequencies_refusals(mol, args, kw):
    with pytest.raises(ValueError):
        mol.rope_frequencies(*args, **kw)


# ---------------------------------------------------------------------------------------- oracle
def test_oracle_rope_hand_worked():
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 5.0]]])
    half = ao.rope(x, [1], [math.pi / 2, math.pi])[0, 0]
    assert half == pytest.approx([-3, -2, 1, -4, 5])
    inter = ao.rope(x, [1], [math.pi / 2, math.pi], True, 2.0)[0, 0]
    assert inter == pytest.approx([-4, 2, -6, -8, 5])


def test_oracle_attention_hand_worked():
    """Two pages of two tokens, keys 0 (so even weights), values 1, 2, 4, 8."""
    k = np.zeros((3, 2, 1, 1))
    v = np.array([[4.0, 8], [100, 100], [1, 2]]).reshape(3, 2, 1, 1)
    q = np.ones((5, 1, 1))
    out, spread, reach = ao.paged_attention(q, k, v, [[2, 0], [2, -1]], [3, 4], [0, 2, 4])
    assert out[:4, 0, 0] == pytest.approx([1.5, 7 / 3, 1.5, 1.5])
    assert np.isnan(out[4]).all()
    out, _, _ = ao.paged_attention(q[:2], k, v, [[2, 0], [2, -1]], [3, 0], None, window=2)
    assert out[:, 0, 0] == pytest.approx([3.0, 0.0])


def test_oracle_append_hand_worked():
    k = np.arange(3.0).reshape(3, 1, 1) + 1
    kc, vc = ao.cache_append(k, -k, np.zeros((2, 2, 1, 1)), np.zeros((2, 2, 1, 1)), [3, -1, 4])
    assert kc.ravel().tolist() == [0, 0, 0, 1] and vc.ravel().tolist() == [0, 0, 0, -1]
