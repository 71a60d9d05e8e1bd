"""The committed records that bench.py reports beside its own measurements."""
import json
import os

import bench


def test_dram_traffic_is_of_the_current_attention_kernels():
    """bench.py reports a recorded DRAM traffic only while the attention kernels' sources are those it was
    captured on: whoever changes them captures it anew, or every line loses its traffic without a word."""
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        recorded = [k for k in json.load(f) if not k.startswith("_")]
    assert sorted(recorded) == ["c1", "c2", "c3", "c4", "c5"]
    for name in recorded:
        assert bench.recorded_traffic(name) is not None, name
