"""The benchmark reports a workload's DRAM bytes only where its committed capture was
taken with the GEMM kernels' present sources: a change of those comes with new
captures.  Runs on the CPU."""
import json

import pytest

import bench

pytestmark = pytest.mark.cpu


def test_captures_are_of_the_present_sources():
    with open(bench.TRAFFIC_FILE) as f:
        records = json.load(f)
    for name, r in records.items():
        kind = "kg" if name.startswith("kgrouped") else "fwd"
        assert r["sources_sha256"] == bench.kernel_sources_sha(kind), name
        assert bench.measured_traffic(name, kind) == r["bytes_per_step"]
