"""CPU checks of how the experts and the 4-bit linear deal out their work: the host side that plans a
launch, compiled by itself (tests/host/moe_plan.cu), over the shapes of the GPU tests and over random
ones of the whole contract."""

import math
import os
import random
import re
import subprocess

import pytest

from tests import test_gpu_block, test_gpu_block_paths
from tests.test_abi_cpu import needs_nvcc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
GATE_UP, DOWN, LINEAR, PAIRS = 0, 1, 2, 3  # of a launch


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    """launches(lines): for each call the launches it makes, as dicts."""
    from moe_lora_virtual_gb300.build import ARCH_FLAGS, nvcc_path

    exe = str(tmp_path_factory.mktemp("plan") / "moe_plan")
    subprocess.run([nvcc_path(), "-std=c++17", "-O1", *ARCH_FLAGS, "-I", os.path.join(ROOT, "include"),
                    "-I", os.path.join(ROOT, "moe_lora_virtual_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "host", "moe_plan.cu"), "-o", exe], check=True)

    def launches(lines):
        out = subprocess.run([exe], input="\n".join(lines), capture_output=True, text=True, check=True)
        out = out.stdout.splitlines()
        assert len(out) == len(lines)
        return [[{k: int(v) for k, v in re.findall(r"(\w+)=(-?\d+)", launch)}
                 for launch in re.findall(r"{(.*?)}", line)] for line in out]

    return launches


def tiles(a):
    return 1 if a["xrows"] <= 8 else 2 if a["xrows"] <= 16 else 4


def way(a):
    """What tells the ways through a kernel apart, of one launch."""
    w4 = a["group"] != 0
    if a["mode"] == DOWN:
        return "down", w4, a["cluster"], a["ksteps"] > 1, tiles(a)
    return ("gate_up", "", "linear", "split")[a["mode"]], w4, a["xstages"], a["chunks"], \
        a["ksteps"] > 1, tiles(a), a["parts"] > 1


def calls_of_the_gpu_tests():
    shapes = list(test_gpu_block_paths.EXPERTS)
    for T, E, k, H, I, _ in test_gpu_block.SHAPES:
        shapes += [(group, T, k, E, H, I) for group in test_gpu_block.FORMATS]
    lines = [f"{half} " + " ".join(map(str, s)) for s in shapes for half in ("gate_up", "down", "split")]
    linear = list(test_gpu_block_paths.LINEAR)
    for mark in test_gpu_block.test_linear.pytestmark:
        if mark.name == "parametrize" and mark.args[0] == "T,K,N":
            linear += [(group, *s) for s in mark.args[1] for group in (32, 64, 128)]
    assert len(linear) > len(test_gpu_block_paths.LINEAR)
    return lines + ["linear " + " ".join(map(str, s)) for s in linear]


def random_calls(n, seed, most=math.inf):
    rng = random.Random(seed)

    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    lines = []
    while len(lines) < n:
        T = log(1, 128)
        k, E, H, I = log(1, 1024 // T), log(1, 1024), 8 * log(1, 8192), 8 * log(1, 8192)
        group = rng.choice([0, 32, 64, 128])
        if 3 * E * H * I <= most and k <= (E if most < math.inf else k):
            lines += [f"{half} {group} {T} {k} {E} {H} {I}" for half in ("gate_up", "down", "split")]
        N = log(1, 1 << 30) if rng.random() < 0.05 else log(1, 200000)
        if group and H * N <= most:
            lines.append(f"linear {group} {log(1, 64)} {H} {N}")
    return lines


@needs_nvcc
def test_the_gpu_tests_reach_every_way(plan):
    """Ways of random shapes of up to 10^9 weights, each expert at most once a token."""
    reached = {way(a) for line in plan(calls_of_the_gpu_tests()) for a in line}
    lines = random_calls(40000, 1, most=1e9)
    missing = {}
    for line, launches in zip(lines, plan(lines)):
        for a in launches:
            if way(a) not in reached:
                missing.setdefault(way(a), line)
    assert not missing, missing


@needs_nvcc
def test_an_entry_a_launch_where_rows_pass_32_bits(plan):
    """Each launch's tokens follow those of the one before, and none is left out."""
    base = 1 << 40
    lines = [f"linear {group} {T} {K} {N}" for group in (32, 64, 128) for T in (33, 50, 64)
             for K in (8, 2048, 20000) for N in (1 << 27, (1 << 30) // 3, (1 << 30) - 15, 1 << 30)]
    several = 0
    for line, launches in zip(lines, plan(lines)):
        _, _, T, K, N = line.split()
        at = 0
        for a in launches:
            assert a["x"] == base + 2 * int(K) * at and a["out"] == base + 2 * int(N) * at, line
            entries = -(-a["tokens"] // a["xrows"])
            assert entries * a["entry_rows"] <= (1 << 30) + 4096, line
            at += a["tokens"]
        assert at == int(T), line
        several += len(launches) > 1
    assert several > len(lines) // 4


def scratch(a):
    """Bytes that grouping the pairs takes: ids, and counts of 16 bits of each warp and expert."""
    numel = a["tokens"] * a["topk"]
    if numel <= 32:
        return 0
    rounds = -(-numel // 512)
    warps = -(-numel // (32 * rounds))
    return 4 * numel + -(-2 * warps * a["E"] // 4) * 4


@needs_nvcc
def test_shared_memory_of_a_launch(plan):
    """The parts of a block's shared memory lie one behind the other and fit; the scratch that groups
    the pairs ends before the lists that it makes: in down it may reach past the ring into the teams'
    sums, which are zeroed afterwards."""
    room = 222 * 1024
    lines = random_calls(60000, 2) + [f"down 0 128 8 1000 1024 {I}" for I in (32, 40, 48, 56)]
    past_ring = 0
    for line, launches in zip(lines, plan(lines)):
        assert launches or line.startswith("split"), f"refused: {line}"
        for a in launches:
            numel, tokens = a["tokens"] * a["topk"], a["tokens"]
            chunk = 2048 + (16 * 512 // a["group"] if a["group"] else 0)
            if a["mode"] == DOWN:
                ring, sums = a["stages"] * a["stage_bytes"], a["teams"] * tokens * a["acc_stride"] * 4
                each = -(-tokens // a["cluster"])
                lists = ring + sums + (each * a["cluster"] * a["acc_stride"] * 4 if a["cluster"] > 1 else 0)
                end, free = lists + 16 * numel, ring + sums
                past_ring += scratch(a) > ring
                assert a["stages"] % a["teams"] == 0 and a["stage_bytes"] >= a["x_off"] + a["xrows"] * a["x_pitch"]
            else:
                warps = 15 if tiles(a) == 4 else 16
                free = warps * a["chunks"] * chunk + a["xstages"] * a["xslot_bytes"]
                end = free + a["teams"] * (a["parts"] - 1) * tiles(a) * 512
                end += 0 if a["mode"] == LINEAR else 12 * numel
                assert a["teams"] * a["parts"] <= warps and a["xslot_bytes"] >= a["xrows"] * a["x_pitch"]
            assert end <= a["smem"] <= room, line
            assert a["mode"] == LINEAR or scratch(a) <= free, line
    assert past_ring >= 4


@needs_nvcc
def test_the_linears_entries(plan):
    """Long rows of many tokens: entries of 8 where their whole rows fit, else pieces of the rows of 16
    (of up to 32 with many outputs). Entries of 4 would read the weights up to 16 times."""
    lines = [f"linear {group} {T} {K} {N}" for group in (32, 64, 128) for T in (9, 16, 24, 33, 48, 64)
             for K in (5000, 8192, 12000, 16384, 65536) for N in (300, 5000, 20000)]
    for line, launches in zip(lines, plan(lines)):
        for a in launches:
            assert a["xrows"] >= 8, line
            assert a["ksteps"] > 1 or a["K"] * 2 * a["xrows"] < 222 * 1024, line
            assert a["ksteps"] == 1 or a["xrows"] >= min(16, a["tokens"]), line
