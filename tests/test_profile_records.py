"""The committed traffic record of the forward kernel belongs to the sources
that are built: a record of other sources is none, and the benchmark's roofline
would go without."""
import json
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import bench  # noqa: E402

with open(os.path.join(ROOT, "profiles", "attn_fwd_traffic.json")) as f:
    RECORD = json.load(f)


@pytest.mark.parametrize("workload", list(RECORD["per_launch_bytes"]))
def test_forward_traffic_is_of_these_sources(workload):
    bytes_, how = bench.profiled_traffic(workload)
    assert bytes_ == RECORD["per_launch_bytes"][workload]["bytes"], how
