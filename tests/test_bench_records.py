"""The counter records that the benchmark's traffic figure comes from were taken
on the present sources: an edit of those, a comment too, leaves the figure empty
until the records are retaken (the commands stand in the profile)."""
import pytest

import bench
from synth import CONFIGS


@pytest.mark.parametrize("workload,row_block", [("stack", 32), ("skew", 32), ("wide", 128)])
def test_traffic_record_is_current(workload, row_block):
    rec = bench.measured_traffic(bench.traffic_key(CONFIGS[workload], "tiled", row_block))
    assert rec is not None
    want = (rec["fetch_kib"] * rec["fetch_factor"] + rec["write_kib"] * rec["write_factor"]) * 1024
    assert abs(rec["bytes_per_launch"] - want) <= 1e-4 * want
    assert rec["bytes_per_launch"] >= rec["algorithmic_bytes"]
