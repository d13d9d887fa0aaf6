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


def test_a_stage_is_refilled_only_behind_its_own_loads():
    """A load from shared memory may come later than a copy by TMA that was asked for behind it: the copy's addresses have to
    hang on what each lane loaded from the stage."""
    s = source("cache_mma.cuh")
    loop = s[s.index("for (int x = 0; x < n_slices; ++x)"):]
    refill = re.search(r"issue\(y, stage,[^;]*;", loop)[0]
    assert re.search(r"__any_sync\(~0u, come\b", refill) and "p.splits" in refill
    assert loop.count("issue(") == 1
    values = re.findall(r"const uint[24] u = lds\w+\(at[^;]*;(.*?)\}", loop, re.S)
    assert len(values) == 2 and all("come |= u.x" in v for v in values)
    assert loop.index("= lds64(at") < loop.index("h == C::NH - 1) refill();") < loop.index("mma_f16(o[")
    issue = re.search(r"auto issue = \[&\]\(([^)]*)\) \{\s*const uint32_t bar = ([^,]*), dst = ([^;]*);", s)
    assert "hold" in issue[1] and "hold" in issue[2] and "hold" in issue[3]


def test_shared_arrays_read_in_fours_are_declared_aligned():
    """Arrays of single words in shared memory that are accessed 16 bytes at a time start on 16 bytes by their declaration, not
    by where the compiler happens to put them."""
    found = set()
    for name in sorted(f for f in os.listdir(CSRC) if f.startswith("cache_")):
        s = source(name)
        alias = dict(re.findall(r"\*\s*(\w+) = (s_\w+)\[", s))
        wide = {alias.get(x, x) for x in re.findall(r"reinterpret_cast<(?:const )?(?:uint4|float4|int4) \*>\((\w+)", s)}
        for align, array in re.findall(r"__shared__ (__align__\(16\) )?(?:unsigned|int|float|uint32_t) ([^;]*);", s):
            for x in re.findall(r"(\w+)\[", array):
                if x in wide:
                    found.add(x)
                    assert align, (name, x)
    assert "s_hist" in found
