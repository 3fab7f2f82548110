"""The DRAM traffic that the benchmark reports beside its roofline was recorded
from the kernels and host code of this tree (no GPU)."""
from __future__ import annotations

import json
import os

import bench

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_recorded_traffic_is_of_these_sources():
    with open(os.path.join(ROOT, "profiles", "traffic.json")) as f:
        record = json.load(f)
    for name, e in record["kernels"].items():
        assert bench.recorded_traffic(name) == e["dram_bytes_per_launch"] == e["dram_read"] + e["dram_write"], name
        # writes may stay in L2; nothing is read or written twice
        assert 0.5 * e["algorithmic_bytes"] < e["dram_bytes_per_launch"] < 1.01 * e["algorithmic_bytes"], name
