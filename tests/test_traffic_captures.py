"""The benchmark's DRAM traffic comes from committed ncu captures of the fused
kernel: each belongs to the code as it is."""
import importlib.util
import json
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

with open(os.path.join(ROOT, "profiles", "ncu_traffic.json")) as f:
    CAPTURES = json.load(f)


@pytest.fixture(scope="module")
def bench():
    spec = importlib.util.spec_from_file_location("bench", os.path.join(ROOT, "bench.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("workload", sorted(CAPTURES))
def test_capture_is_of_this_code(bench, workload):
    traffic, source = bench.ncu_traffic(workload)
    assert traffic == CAPTURES[workload]["bytes_per_launch"], source
