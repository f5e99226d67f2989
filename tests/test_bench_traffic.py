"""The DRAM traffic that the bench reports beside its rooflines was recorded on the present kernel sources."""
import json
import os

import pytest

import bench

with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
    RECORDED = json.load(f)


@pytest.mark.parametrize("name", sorted(n for n in RECORDED if n.startswith("tc_")))
def test_recorded_traffic_belongs_to_the_present_sources(name):
    kernel, workload = name.split(":")
    assert bench.measured_traffic(kernel, workload, bench.KERNEL_SOURCES[kernel]) == RECORDED[name]["dram_bytes_per_launch"]
