"""How sq_kvq_attention cuts a call, on the host: its workspace is never more than the size
that callers are told, for the same sizes or smaller ones, with a window or without."""
import os
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
LIBDIR = os.path.join(os.path.dirname(HERE), "quantized_recurrent_state_gated_amd")


@pytest.fixture(scope="module")
def fuzz(tmp_path_factory):
    out = str(tmp_path_factory.mktemp("plan") / "fuzz")
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    os.path.join(HERE, "kvq_plan_fuzz.cpp"), "-o", out, f"-L{LIBDIR}", "-lsq", f"-Wl,-rpath,{LIBDIR}",
                    "-L/opt/rocm/lib", "-lamdhip64", "-Wl,-rpath,/opt/rocm/lib"], check=True)
    return out


@pytest.mark.parametrize("seed", [1, 2, 3, 4])
def test_calls_need_no_more_than_their_workspace(fuzz, seed):
    r = subprocess.run([fuzz, str(seed), "500000"], capture_output=True, text=True, timeout=100)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "with a workspace" in r.stdout
