"""A kernel of the adapters whose bounded wait gives up leaves no copy and no tensor-core product in
flight: it waits for them behind the block's last barrier, where no role can give up any more, and not
only in the role that gave up itself.  (A source check: a wait that runs out is not provoked.)"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "grouped_expert_gemm_gb300", "csrc")


@pytest.mark.parametrize("name", ["adapter_project.cuh", "adapter_shrink.cu", "adapter_grads.cu"])
def test_everything_in_flight_is_waited_for_behind_the_roles(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    waits = [m.start() for m in re.finditer(r"wait_bounded", text)]
    drains = [m.start() for m in re.finditer(r"wait_drain\(", text)]
    assert waits and len(drains) >= 2 and drains[0] > waits[-1]
    between = text[waits[-1]:drains[0]]
    barrier = between.rindex("__syncthreads();")
    assert "*abort_flag" in between[barrier:] and "!ok" not in between[barrier:]
    assert re.search(r"wait_drain\(full_bar\(", text) and re.search(r"wait_drain\(drain_bar", text)
