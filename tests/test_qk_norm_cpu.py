"""Norms and rotation of queries and keys: what the source has to keep to."""

import os
import re

from token_weight_scans_b200 import build


def test_rows_that_may_be_written_in_place_are_read_by_plain_loads():
    """dq and dk may be q and k. The read-only data path (__ldg, ld.global.nc, __restrict__) is for
    memory that no thread of the kernel writes: the compiler may repeat such a load after a store."""
    with open(os.path.join(build.CSRC, "qk_norm_rope.cu")) as f:
        source = re.sub(r"//[^\n]*", "", f.read())
    for word in ("__ldg", "ld.global.nc", "__restrict__"):
        assert word not in source
