"""The benchmark reports the selection kernel's DRAM traffic from the committed captures, which hold for the source
that they were taken on: a change of one of its files asks for new captures, and helpers of other
kernels belong into files of their own."""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)


@pytest.mark.parametrize("workload", ["h128k", "h128k-e4m3"])
def test_the_captured_traffic_is_the_present_sources(workload):
    import bench
    src = bench.source_hash("select_kernel.cuh", "attn_core.cuh", "common.cuh")
    got = bench.traffic_for("select_kernel", workload, src)
    assert got is not None and got > 0
