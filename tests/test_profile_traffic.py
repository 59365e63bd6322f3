"""The DRAM traffic that bench.py reports was taken on the forward's present
sources: files that the forward shares with other operators count too."""
import json
import os

import pytest

import bench
import seeded_inputs

NAMES = [w["name"] for w in
         seeded_inputs.WORKLOADS + seeded_inputs.KV_WORKLOADS + seeded_inputs.VARLEN_WORKLOADS]


@pytest.mark.parametrize("name", NAMES)
def test_traffic_is_of_the_present_sources(name):
    traffic, note = bench.stored_traffic(name)
    assert traffic is not None and traffic > 0, note


def test_captures_add_up():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        data = json.load(f)
    assert sorted(data["workloads"]) == sorted(NAMES)
    for entry in data["workloads"].values():
        assert entry["dram_bytes_per_launch"] == entry["dram_read"] + entry["dram_write"]
        assert entry["kernel_hash"] == data["kernel_hash"] == bench.kernel_source_hash()
