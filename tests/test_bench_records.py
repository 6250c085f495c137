"""The benchmark's recorded HBM traffic belongs to the sources that are here: a
change to one of them makes its traffic unknown until it is taken again."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bench  # noqa: E402


@pytest.mark.parametrize("name", sorted(bench.COUNTERS))
def test_traffic_is_known(name):
    traffic = bench.measured_traffic(name)
    assert traffic is not None, f"{name}: the sources changed since its counters were taken"
    assert traffic > 5e8
