"""Build libozaki2.so (HIP, gfx950) in-tree with hipcc.

Usage: python -m rns_emulated_fp64_amd.build
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libozaki2.so")
SOURCES = ["kernels.hip", "api.cpp", "tables.cpp", "noalloc.hip", "products.hip", "xent.hip", "norm.hip", "linear.hip", "sample.hip"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    # exact integer arithmetic in doubles: never contract a*b+c behind our back
    "-ffp-contract=off",
    # no packed FP32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    err = "\n".join(l for l in res.stderr.splitlines() if "packed-fp32-ops" not in l)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed ({res.returncode}):\n{err}")


def build(verbose: bool = False) -> str:
    """Every source is compiled anew, several at a time, and linked into LIB, which appears only when whole."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as objects:
        outs = [os.path.join(objects, s + ".o") for s in SOURCES]
        cmds = [[hipcc, *[f for f in HIPCC_FLAGS if f != "-shared"], "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-c",
                 os.path.join(CSRC, s), "-o", o] for s, o in zip(SOURCES, outs)]
        with concurrent.futures.ThreadPoolExecutor(min(len(cmds), 8)) as pool:
            list(pool.map(lambda cmd: _run(cmd, verbose), cmds))
        _run([hipcc, "--offload-arch=gfx950", "-shared", "-fPIC", *outs, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
