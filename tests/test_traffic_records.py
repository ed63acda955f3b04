"""The DRAM traffic that bench.py reports comes from counted launches, as long as the sources are those counted."""
import json
import os

import pytest

import bench
from block_sparse_attention_qp_gb300.inputs import WORKLOADS

with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
    RECORDS = json.load(f)


@pytest.mark.parametrize("kernel", sorted(RECORDS))
def test_record_is_of_these_sources(kernel):
    """A change to a counted kernel's sources leaves the bench line without its traffic: count the launches again (the
    command stands beside the figures) and put down the sources' new hash."""
    r = RECORDS[kernel]
    assert r["src_hash"] == bench.src_hash(*r["src_files"])
    w = next(w for w in WORKLOADS if w.name == r["workload"])
    assert bench.traffic_record(kernel, w) == r["dram_bytes_read"] + r["dram_bytes_write"] > 0
