"""The block's kernels may be on the GPU before the kernel that writes their inputs has ended (programmatic dependent launch), so none of
them reads through the read-only path, whose loads may be moved before the wait: it is for data that nobody writes meanwhile."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_quantised_gb300", "csrc")
FILES = [f for pattern in ("woq_block_*", "woq_route.cu", "woq_experts*") for f in sorted(glob.glob(os.path.join(CSRC, pattern)))]


@pytest.mark.parametrize("path", FILES, ids=[os.path.basename(f) for f in FILES])
def test_no_read_only_loads(path):
    with open(path) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__ldg\b|\.nc\b|__restrict__", code)
