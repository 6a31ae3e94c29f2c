"""The HBM traffic that bench.py reports comes from counters of the committed
kernels: the summaries under profiles/ hold the hash of the sources that they
were taken from, and it is that of the sources here. (A change of the single
pass, its launcher or the compile flags takes new counters.)"""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.mark.parametrize("workload", ["7p5b", "llama8b", "70b"])
def test_counters_are_those_of_the_sources(workload):
    traffic = bench.read_traffic(workload, "k_fused", bench.source_hash("k_fused"))
    assert traffic is not None and traffic > 1e9


def test_counters_of_other_sources_are_not_reported():
    assert bench.read_traffic("7p5b", "k_fused", "0" * 16) is None
    assert bench.read_traffic("gpt2", "k_fused", bench.source_hash("k_fused")) is None  # none were taken
