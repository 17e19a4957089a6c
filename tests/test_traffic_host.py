"""The DRAM bytes kept with the profiles are those of the sources as they are: bench.py reports none for a
kernel whose sources have changed since, so a record that no longer fits is retaken or taken out."""
import json
import os

import bench


def test_every_record_is_of_the_current_sources():
    with open(os.path.join(bench.ROOT, "profiles", "traffic.json")) as f:
        table = json.load(f)
    stale = [k for k, rec in table.items() if rec["source_hash"] != bench.kernel_source_hash(rec["kernel"])]
    assert not stale
    for key, rec in table.items():
        assert bench.measured_traffic(key.split(":")[0], rec["kernel"]) == rec["dram_bytes_per_launch"]
        assert os.path.exists(os.path.join(bench.ROOT, "profiles", rec["profile"]))
