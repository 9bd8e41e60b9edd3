"""Rules of the hardware that no run shows broken, read off the source (CPU)."""
import os
import re

import sparse_attention_token_index_b200 as dsa


def _kernel():
    with open(os.path.join(os.path.dirname(dsa.__file__), "csrc", "dsa_attend_tc.cu")) as f:
        return f.read()


def test_a_warpgroup_changes_its_registers_by_one_instruction():
    # setmaxnreg is undefined where the warps of a warpgroup execute different ones: each share is set in one place, ahead
    # of any branch that tells the group's warps apart
    shares = re.findall(r"set_regs<C::(\w+)", _kernel())
    assert sorted(shares) == ["kCopyRegs", "kMidRegs", "kSoftRegs"]
