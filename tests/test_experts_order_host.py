"""What orders the experts' kernels' shared memory between lanes, read from their
source (no GPU): a missing wait shows in no result while the hardware happens to
issue in order."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_quantized_qgemm_gb300", "csrc")


def code_lines(name):
    """The file's lines without comments and blank ones."""
    with open(os.path.join(CSRC, name)) as f:
        lines = [re.sub(r"//.*", "", line).strip() for line in f]
    return [line for line in lines if line]


@pytest.mark.parametrize("barrier,places", [("sempty(", 2), ("to_issuer", 2)])
def test_lanes_meet_before_one_of_them_gives_a_slot_back(barrier, places):
    """An arrival orders the reads of the lane that makes it.  A slot that all
    lanes read (of activation scales; of accumulators) is given back behind a
    __syncwarp, in both forms of the grouped GEMM."""
    lines = code_lines("qg_grouped.cu")
    at = [i for i, line in enumerate(lines) if re.search(r"\barrive(_cluster)?_if\(lane == 0, " + re.escape(barrier), line)]
    assert len(at) == places
    for i in at:
        while "arrive" in lines[i]:   # the forms' arrivals stand below one another
            i -= 1
        assert lines[i] == "__syncwarp();", lines[i]
