"""CPU checks of the MoE block's kernels and of the host code around them."""

import os
import re
import shutil
import subprocess

import pytest

from tests.test_abi_cpu import needs_nvcc

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_lora_virtual_gb300", "csrc")


def cuda_include():
    from moe_lora_virtual_gb300.build import nvcc_path

    return os.path.join(os.path.dirname(os.path.dirname(nvcc_path())), "include")


needs_gcc = pytest.mark.skipif(not shutil.which("g++"), reason="g++ not available")


def test_waits_of_the_streaming_kernels_are_the_warps():
    """Every wait there is taken by a whole warp, whose lanes have to agree on its outcome: a poll of
    its own decides for no lane."""
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "mol_moe.cuh")).read())
    assert len(re.findall(r"\bwarp_wait\(", code)) > 1
    assert re.findall(r"[^\n;{]*\bmbar_(?:try_)?wait\([^\n]*", code) == [
        "  return __all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitPolls, limit_ns));"]


@needs_nvcc
@needs_gcc
def test_the_experts_kernels_are_prepared_for_their_own_calls(tmp_path):
    """Where they cannot be prepared (a down block takes all of an SM's shared memory) the LoRA path,
    the norm and the router's choice go on; elsewhere each set of kernels is prepared once."""
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "mol_lora.cu")).read())
    assert "prepare_moe_kernels" not in src
    exe = str(tmp_path / "device_state")
    subprocess.run(["g++", "-O1", "-std=c++17", "-no-pie", "-I", os.path.join(ROOT, "include"), "-I",
                    CSRC, "-I", cuda_include(), "-x", "c++", os.path.join(CSRC, "mol_abi.cu"),
                    os.path.join(CSRC, "mol_block_abi.cu"),
                    os.path.join(ROOT, "tests", "host", "device_state.cpp"), "-o", exe,
                    # the launchers of calls that the program does not make
                    "-Wl,--unresolved-symbols=ignore-all"], check=True)
    assert subprocess.run([exe], capture_output=True, text=True).stdout == "ok\n"
