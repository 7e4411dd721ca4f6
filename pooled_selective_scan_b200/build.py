"""Build ``libfastvim_ssm.so`` in-tree with nvcc for sm_100a (B200).

    python -m pooled_selective_scan_b200.build [--force] [--verbose]

The library is plain CUDA C++ behind a C ABI (``include/fastvim_ssm.h``); nvcc cross-compiles it
without a GPU.  The CUDA runtime is linked statically, so the library does not depend on the
runtime version a host process (e.g. PyTorch) carries.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libfastvim_ssm.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
]
LINK_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static"]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the FastVim SSM library needs the CUDA toolkit to build")


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def needs_build() -> bool:
    if not os.path.exists(LIB_PATH):
        return True
    t = os.path.getmtime(LIB_PATH)
    return any(os.path.getmtime(s) > t for s in sources())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not needs_build():
        return LIB_PATH
    nvcc = nvcc_path()
    units = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with tempfile.TemporaryDirectory(dir=PKG, prefix="_build") as tmp:
        objs = [os.path.join(tmp, os.path.basename(u)[:-3] + ".o") for u in units]
        flags = [*(["-Xptxas=-v"] if verbose else []), *NVCC_FLAGS, "-I" + INCLUDE, "-I" + CSRC]
        with ThreadPoolExecutor(max_workers=max(1, min(len(units), os.cpu_count() or 1))) as pool:
            list(pool.map(lambda uo: _run([nvcc, *flags, "-c", "-o", uo[1], uo[0]], verbose), zip(units, objs)))
        lib = os.path.join(tmp, LIB_NAME)
        _run([nvcc, *LINK_FLAGS, "-o", lib, *objs], verbose)
        os.replace(lib, LIB_PATH)
    return LIB_PATH


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=not verbose, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{(res.stderr or '') + (res.stdout or '')}")


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))
    return 0


if __name__ == "__main__":
    sys.exit(main())
