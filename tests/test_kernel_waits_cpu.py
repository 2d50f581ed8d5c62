"""The order of waits in the sources of the experts' products, without a GPU.

Loads straight into LDS are counted as vector memory operations of the wave that
issues them: a barrier alone orders nothing there.  So between such a load and
the next barrier, behind which other waves read what it wrote, a wait of the
issuing wave has to stand."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "combine_balanced_planning_amd", "csrc", "moon_expert.hip")


def kernel(name):
    """Text of a kernel, to the next one or the host code, without comments."""
    with open(SOURCE) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index(name + "(ExpertArgs")
    ends = [text.find(e, at) for e in ("__global__", "moon_status check(")]
    return text[at:min(e for e in ends if e > 0)]


@pytest.mark.parametrize("name", ["k_expert_stream", "k_expert_tiles"])
def test_lds_loads_are_waited_for(name):
    events = re.findall(r"\bfill(?:_scales)?\(|\bwait_vm<|__syncthreads\(|amdgcn_s_barrier\(", kernel(name))
    assert sum(e.startswith("fill") for e in events) >= 4
    pending = False
    for i, e in enumerate(events):
        if e.startswith("fill"):
            pending = True
        elif e == "wait_vm<":
            pending = False
        else:
            assert not pending, f"{name}: barrier {i} of {events} behind loads that nothing waits for"
    assert not pending, f"{name}: loads may land in LDS after the workgroup has left"
