"""The kernel instances that bench.py reports and picks out of profiles are
instances of the built library, under the names that a profiler prints."""
import json
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


@pytest.fixture(scope="module")
def names():
    lib = os.path.join(ROOT, "quantized_recurrent_state_gated_amd", "libsq.so")
    out = subprocess.run(["nm", "-C", lib], capture_output=True, text=True, check=True).stdout
    return {line.split(" void sqk::", 1)[1].split("(")[0] for line in out.splitlines() if " void sqk::k_" in line}


@pytest.mark.parametrize("kda", [False, True])
@pytest.mark.parametrize("tiles", [1, 1023, 1024, 16383, 16384, 70 * 2304])
def test_reported_instances_exist(names, tiles, kda):
    assert bench.step_kernel(tiles, kda) in names


def test_counted_instances_exist(names):
    assert bench.STEP_KERNEL in names and bench.KDA_KERNEL in names
    assert bench.step_kernel(70 * 2304) == bench.STEP_KERNEL
    assert bench.step_kernel(70 * 2304, kda=True) == bench.KDA_KERNEL


@pytest.mark.parametrize("workload", ["serving", "highconc"])
def test_committed_counters_are_of_these_instances(workload):
    with open(bench.traffic_file(workload)) as f:
        t = json.load(f)
    assert t["step"]["kernel"] == bench.STEP_KERNEL
    assert t["channel_gate_step"]["kernel"] == bench.KDA_KERNEL
