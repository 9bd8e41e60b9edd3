"""Rules of the hardware that no run shows broken, read off the source (CPU)."""
import os
import re

import sparse_attention_token_index_b200 as dsa


def _kernel(name="dsa_attend_tc.cu"):
    with open(os.path.join(os.path.dirname(dsa.__file__), "csrc", name)) as f:
        return f.read()


def test_a_warpgroup_changes_its_registers_by_one_instruction():
    # setmaxnreg is undefined where the warps of a warpgroup execute different ones: each share is set in one place, ahead
    # of any branch that tells the group's warps apart
    shares = re.findall(r"set_regs<C::(\w+)", _kernel())
    assert sorted(shares) == ["kCopyRegs", "kMidRegs", "kSoftRegs"]


def test_the_debug_build_checks_the_paged_kernels():
    # each site has a number of its own
    sites = []
    for name in ("dsa_paged.cuh", "dsa_attend.cu", "dsa_attend_tc.cu", "dsa_pages.cu"):
        found = re.findall(r"in_bounds\(.*?a\.status, (\d+)\)", _kernel(name), re.S)
        assert found, name
        sites.append({int(x) for x in found})
    assert sum(map(len, sites)) == len(set.union(*sites)) and min(set.union(*sites)) >= 20
