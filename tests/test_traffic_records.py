"""The recorded DRAM bytes that the bench line reports belong to the kernels as they are now (CPU only).
After a change to one of their sources: capture again with the entry's command, then bench.py --record-traffic."""
import importlib.util
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
with open(os.path.join(ROOT, "profiles", "dram_traffic.json")) as f:
    ENTRIES = json.load(f)["entries"]


@pytest.mark.parametrize("key", sorted(ENTRIES))
def test_record_is_of_the_present_sources(key):
    spec = importlib.util.spec_from_file_location("bench_records", os.path.join(ROOT, "bench.py"))
    bench = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(bench)
    assert bench.measured_traffic(key) == ENTRIES[key]["dram_bytes_per_launch"]
