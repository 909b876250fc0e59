"""Build ``libfa_sm100.so`` (the C-ABI attention library) in-tree with nvcc for sm_100a.

The library is two translation units, ``csrc/fa_api.cu`` and ``csrc/fa_api_score.cu``, which
include the kernels and are compiled side by side.
It links the CUDA runtime statically and reaches the driver's tensor-map encoder through
``cudaGetDriverEntryPoint``, so it needs no link-time driver library.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libfa_sm100.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-v",
]
UNITS = ["fa_api.cu", "fa_api_score.cu"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h")) + [os.path.join(INCLUDE, "fa.h")])


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library if missing or older than any source; return its path."""
    if not force and os.path.exists(LIB):
        newest = max(os.path.getmtime(s) for s in _sources())
        if os.path.getmtime(LIB) >= newest:
            return LIB
    jobs = []
    with tempfile.TemporaryDirectory() as tmp:
        for unit in UNITS:
            obj = os.path.join(tmp, unit + ".o")
            cmd = [_nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, unit), "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            log = open(os.path.join(tmp, unit + ".log"), "w+")
            jobs.append((obj, log, subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT)))
        logs, failed = [], False
        for obj, log, job in jobs:
            failed = job.wait() != 0 or failed
            log.seek(0)
            logs.append(log.read())
            log.close()
        if failed:
            raise RuntimeError("nvcc failed:\n" + "".join(logs))
        cmd = [_nvcc(), *NVCC_FLAGS[:2], "-Xcompiler", "-fPIC", "-shared", *(j[0] for j in jobs), "-o", LIB + ".tmp"]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    with open(os.path.join(HERE, "ptxas_resources.txt"), "w") as f:
        f.write("".join(logs))
    os.replace(LIB + ".tmp", LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
