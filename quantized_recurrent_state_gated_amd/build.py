"""Build libsq.so (the HIP kernels + C ABI) in-tree for gfx950.

    python -m quantized_recurrent_state_gated_amd.build [-v]

Packed-FP32 instructions are disabled for all device code.  The sources are
compiled side by side, at most MAX_JOBS (or 8) at a time, and linked.
"""
import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libsq.so")
SOURCES = ["sq_kernels.hip", "sq_api.hip", "sq_paged.hip", "sq_prefill.hip", "sq_serve_api.hip",
           "sq_kvq.hip", "sq_kvq_few.hip", "sq_kvq_tiles.hip", "sq_kvq_api.hip"]
ARCH = os.environ.get("SQ_OFFLOAD_ARCH", "gfx950")


def hipcc_cmd(out: str, *args: str) -> list:
    return (["/opt/rocm/bin/hipcc", f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
             "-Wall", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-o", out] + list(args))


def _run(cmd: list, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in r.stderr.splitlines() if noise not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed ({r.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, flush=True)


def build(verbose: bool = False) -> str:
    jobs = min(int(os.environ.get("MAX_JOBS", "8")), 8)
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(max(1, jobs)) as pool:
        objs = [os.path.join(tmp, s + ".o") for s in SOURCES]
        list(pool.map(lambda so: _run(hipcc_cmd(so[1], "-c", os.path.join(CSRC, so[0])), verbose), zip(SOURCES, objs)))
        _run(hipcc_cmd(OUT + ".tmp", "-shared", *objs), verbose)
    os.replace(OUT + ".tmp", OUT)
    return OUT


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
