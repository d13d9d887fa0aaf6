"""What the sources of the 8-bit cache's kernels must say for their order to hold, where no run shows it: read on the CPU."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "attention_flash_attn_gb300", "csrc")


def source(name):
    """A file of csrc without its comments."""
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*", "", f.read())


def test_marks_of_nans_are_cleared_by_all_warps_before_any_warp_begins():
    """s_nan and s_any are cleared by all threads and marked by single warps, on each way into the first run: the barrier has to
    stand before the ways part."""
    s = source("cache_mma.cuh")
    cleared = s.index("s_nan[x] = 0u")
    parts = s.index("if (p.cluster)", cleared)
    assert "s_any = 0" in s[cleared:parts] and "__syncthreads()" in s[cleared:parts]
