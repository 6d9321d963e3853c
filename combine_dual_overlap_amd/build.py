"""Builds libdbomoe.so (all HIP kernels + the C ABI) for gfx950 with hipcc.

Run as ``python -m combine_dual_overlap_amd.build``; the library lands next to
this file.  hipcc cross-compiles, so no GPU is needed to build.
"""
import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libdbomoe.so")
SOURCES = ["route.hip", "dispatch.hip", "ffn.hip", "combine.hip", "layer.hip", "grouped_gemm.hip", "backward.hip",
           "adamw.hip", "balance.hip", "int8.hip", "norms.hip"]
ARCH = "gfx950"


def jobs() -> int:
    """Compilers at a time: MAX_JOBS if that is a whole number from 1 on, else the CPUs; at most 8."""
    most = os.environ.get("MAX_JOBS", "").strip()
    return min(8, int(most) if most.isdecimal() and int(most) > 0 else os.cpu_count() or 1)


def hipcc() -> str:
    for c in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found (ROCm is required to build libdbomoe.so)")


def build(verbose: bool = False) -> str:
    """Compile every source, several at a time, and link the shared library; returns its path."""
    cc = [hipcc(), f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
          "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
          "-Wall", "-Wno-unused-function", "-Wno-unused-variable", f"-I{INCLUDE}", f"-I{CSRC}"]

    def run(cmd) -> str:
        r = subprocess.run(cmd, capture_output=True, text=True)
        out = "\n".join(l for l in (r.stdout + r.stderr).splitlines() if "packed-fp32-ops" not in l)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed ({r.returncode}):\n{' '.join(cmd)}\n{out}")
        return out

    if verbose:
        print(" ".join(cc), flush=True)
    with tempfile.TemporaryDirectory() as tmp, ThreadPoolExecutor(jobs()) as pool:
        objects = [os.path.join(tmp, s + ".o") for s in SOURCES]
        outs = list(pool.map(lambda s, o: run(cc + ["-c", os.path.join(CSRC, s), "-o", o]), SOURCES, objects))
        outs.append(run([cc[0], f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", LIB + ".tmp"] + objects))
    if verbose:
        print("\n".join(o for o in outs if o.strip()), flush=True)
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
