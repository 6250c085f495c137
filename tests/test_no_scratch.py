"""No kernel of the library keeps registers in scratch memory: a reload there
waits for every copy in flight, in the middle of a tile.  Read from the kernels'
metadata in the built library (keys and small numbers in MessagePack: a number
below 128 is its own byte)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "dsa_lightning_indexer_03_amd", "libdsaidx.so")


def test_no_kernel_spills():
    if not os.path.exists(LIB):
        pytest.skip("libdsaidx.so not built")
    with open(LIB, "rb") as f:
        data = f.read()
    # (scalar registers spill to lanes of vector ones, not to memory)
    names = [m.group(1).decode() for m in re.finditer(rb"\.name[\xd9\xda].{1,2}?(_ZN6dsaidx\w+)", data, re.S)]
    for key in (rb"\.vgpr_spill_count", rb"\.private_segment_fixed_size"):
        got = [data[m.end()] for m in re.finditer(key, data)]
        assert len(got) == len(names) > 100
        assert not any(got), f"{key}: {[n for n, x in zip(names, got) if x]}"
