"""The stored HBM traffic of the step's kernels belongs to the sources that are there: the
benchmark reports it only then, and its line would silently lose it."""
import glob
import os

import pytest

import bench
from ep_synth.configs import config_by_name

STORED = sorted(os.path.basename(f)[len("traffic_"):-len(".txt")]
                for f in glob.glob(os.path.join(bench.PROFILES, "traffic_*.txt")))


def test_the_workloads_with_stored_traffic():
    assert {"deepseek_prefill", "deepseek_decode", "qwen3_moe", "skewed_fp8"} <= set(STORED)


@pytest.mark.parametrize("name", STORED)
def test_stored_traffic_is_of_the_present_sources(name):
    traffic = bench.stored_traffic(config_by_name(name))
    assert traffic is not None, "the kernels' sources changed: measure the traffic again"
    assert traffic > 1e8
