"""The bench's DRAM figures belong to the sources they were captured on: a changed source drops them, so it wants a new
capture, or the change kept out of these files."""
import os
import sys

import pytest

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bench  # noqa: E402


@pytest.mark.parametrize("kernel,workloads", list(bench.TRAFFIC))
def test_captured_traffic_is_of_the_present_sources(kernel, workloads):
    for wl in workloads:
        assert bench.traffic_for(kernel, wl) == bench.TRAFFIC[kernel, workloads][2]
