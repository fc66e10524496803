"""CPU: the router, the route lists and the combine read results of the kernel
before them, beside which they may have been started.  Their sources keep to
loads that cannot move above the wait for it: no read-only or cache-hinted
intrinsic, and no const __restrict__ argument, whose loads the compiler may
turn into read-only ones."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "routed_expert_ffn_02_gb300", "csrc")


@pytest.mark.parametrize("name", ["route.cu", "route_dev.cuh", "permute.cu", "combine.cu", "combine_dev.cuh"])
def test_no_load_that_may_move_above_the_wait(name):
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.findall(r"__ld(?:g|ca|cg|cs|lu|cv)\s*\(", code)
    assert not re.findall(r"const\s+\w+\s*\*\s*__restrict__", code)
