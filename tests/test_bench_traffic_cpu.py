"""The benchmark's DRAM traffic constants are of the sources that are there: a change of a kernel's file without new
counters would drop them from its line (CPU only)."""
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("bench_under_test", os.path.join(ROOT, "bench.py"))


@pytest.fixture(scope="module")
def bench():
    import sys
    m = importlib.util.module_from_spec(spec)
    sys.modules[spec.name] = m
    spec.loader.exec_module(m)
    yield m
    del sys.modules[spec.name]


@pytest.mark.parametrize("key", ["gemm_qwen3", "gemm_gpt2", "adam_gpt2"])
def test_the_constant_is_of_the_source(bench, key):
    assert bench.source_hash(bench.TRAFFIC[key]["source"]) == bench.TRAFFIC[key]["sha256_prefix"]
    assert bench.traffic_for(key) == bench.TRAFFIC[key]["bytes_per_launch"]
