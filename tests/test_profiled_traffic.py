"""The profiled DRAM traffic that the benchmark reports belongs to the kernel
source as it stands.  (A change to that source wants the record taken again, by
the commands in the profile it names; until then the benchmark reports none.)
"""
import json
import os

import pytest

import bench

with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
    RECORDS = json.load(f)


@pytest.mark.parametrize("config", sorted(RECORDS["direct_receive"]))
def test_the_record_is_of_the_current_source(config):
    rec = RECORDS["direct_receive"][config]
    assert bench.profiled_traffic("direct_receive", bench.DR_SOURCES, int(config)) == rec["dram_bytes_per_launch"]
    moved = rec["measured"]["dram_bytes_read"] + rec["measured"]["dram_bytes_write"]
    assert rec["dram_bytes_per_launch"] == moved * 147200 // rec["measured"]["rows"]
