"""Build the reshard library (``libreshard.so``) in-tree for gfx950.

Run ``python -m dtensor_layout_movement_amd.build`` (or call ``build()``).  The
library is always rebuilt: hipcc cross-compiles the gfx950 code object on a
machine without a GPU.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
LIB_PATH = os.path.join(PKG_DIR, "libreshard.so")
SOURCES = [os.path.join(CSRC, f) for f in ("plan.cpp", "kernel.hip", "reshard.hip", "checks.cpp",
                                           "blocks.hip", "block_quantize.hip", "block_matmul.hip", "block_grad.hip",
                                           "groups.hip", "group_quantize.hip", "group_matmul.hip", "group_tiles.hip",
                                           "expert_route.hip")]

# Packed-fp32 instructions are kept out of every HIP object; the copy kernel does
# no floating point and the block-scaled products do theirs on the matrix cores,
# so this costs nothing.
HIP_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-Wall",
    "--offload-arch=gfx950",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    for cand in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the reshard library needs ROCm's hipcc")


def build(verbose: bool = False) -> str:
    """Compile SOURCES, each on its own and several at a time, and link them into
    libreshard.so; return its path."""
    with tempfile.TemporaryDirectory() as folder:
        jobs = []
        for src in SOURCES:
            obj = os.path.join(folder, os.path.basename(src) + ".o")
            jobs.append(([hipcc(), *HIP_FLAGS, "-c", "-I", INCLUDE, "-I", CSRC, src, "-o", obj], obj))
        with ThreadPoolExecutor(_jobs()) as pool:
            list(pool.map(lambda job: _run(job[0], verbose), jobs))
        tmp = LIB_PATH + ".tmp"
        _run([hipcc(), *HIP_FLAGS, "-shared", *[obj for _, obj in jobs], "-o", tmp], verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def _jobs() -> int:
    """Compilers at a time: eight, or fewer where MAX_JOBS is a number of them."""
    given = os.environ.get("MAX_JOBS", "").strip()
    return min(8, int(given) if given.isdecimal() and int(given) else 8)


def _run(cmd, verbose) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass warns that it does not know the packed-fp32 feature; drop that line
    noise = ("packed-fp32-ops", "warning: feature flag")
    msgs = [ln for ln in (res.stdout + res.stderr).splitlines() if not any(n in ln for n in noise)]
    if res.returncode != 0:
        raise RuntimeError("hipcc failed:\n" + "\n".join(msgs))
    if verbose and msgs:
        print("\n".join(msgs), flush=True)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
