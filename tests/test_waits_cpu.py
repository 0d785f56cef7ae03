"""Barrier waits that some lanes of a warp make for all, read from the kernels' sources: a shuffle or a vote passes on the
outcome but orders no memory between the lanes, so a __syncwarp has to follow before what was waited for is used."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_03_b200", "csrc")
FILES = sorted(glob.glob(os.path.join(CSRC, "*.cu*")))


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f) for f in FILES])
def test_a_shared_wait_orders_memory(path):
    lines = [re.sub(r"//.*", "", x) for x in open(path)]
    for i, line in enumerate(lines):
        lane0 = "__shfl_sync" in line and re.search(r"\bok\b", line)
        # lanes at different barriers (or at an earlier look's outcome); a vote on one barrier that every lane has tried
        # itself needs nothing
        split = "__all_sync" in line and re.search(r"\?|\bready\b", line)
        if lane0 or split:
            assert any("__syncwarp()" in x for x in lines[i + 1:i + 5]), "%s:%d" % (path, i + 1)
