"""The counter summaries that bench.py reads belong to the present kernel sources (no GPU needed)."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import bench  # noqa: E402


@pytest.mark.parametrize("workload", ["sasrec", "tenmillion"])
@pytest.mark.parametrize("phase", ["project", "select"])
def test_traffic_is_known(phase, workload):
    """A line of another digest is left out and the traffic reported as unknown: after a change to the phase's sources
    (bench.PHASE_SOURCES) it is measured again."""
    assert bench.measured_traffic(phase, workload) > 0
