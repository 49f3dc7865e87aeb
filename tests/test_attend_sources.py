"""CPU check of the attention kernels' source: where a warp's first lane arrives for all of
them, a barrier of the warp stands before it, which orders the other lanes' reads (a vote
does not)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "few_row_packed_gb300", "csrc")


@pytest.mark.parametrize("name", ["attend_rows.cu", "attend4_rows.cu", "attend_tiles.cuh"])
def test_a_warp_meets_before_its_first_lane_arrives(name):
    with open(os.path.join(CSRC, name)) as f:
        lines = [re.sub(r"//.*", "", line).strip() for line in f]
    lines = [line for line in lines if line]
    found = [i for i in range(len(lines) - 1) if lines[i] == "if (lane == 0)" and lines[i + 1].startswith("mbar_arrive(")]
    assert found
    for i in found:
        assert lines[i - 1] == "__syncwarp();", lines[i - 1:i + 2]
