"""CPU checks of the MoE block's kernels and of the host code around them."""

import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "moe_lora_virtual_gb300", "csrc")


def test_waits_of_the_streaming_kernels_are_the_warps():
    """Every wait there is taken by a whole warp, whose lanes have to agree on its outcome: a poll of
    its own decides for no lane."""
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "mol_moe.cuh")).read())
    assert len(re.findall(r"\bwarp_wait\(", code)) > 1
    assert re.findall(r"[^\n;{]*\bmbar_(?:try_)?wait\([^\n]*", code) == [
        "  return __all_sync(0xffffffffu, mbar_wait(bar, parity, kWaitPolls, limit_ns));"]
