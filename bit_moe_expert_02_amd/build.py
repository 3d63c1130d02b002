"""Builds libmoe.so (HIP kernels for gfx950 + host packer + C ABI) in-tree.

    python -m bit_moe_expert_02_amd.build          # or build() from Python

The library lands next to this file; the binding loads it from there.
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
LIB = os.path.join(HERE, "libmoe.so")

SOURCES = ["moe_kernels.hip", "prefill.hip", "group.hip", "group_gemm.hip", "q4_matvec.hip", "pack.cpp",
           "host_api.cpp", "alloc.cpp", "offload.cpp", "group_host.cpp"]
HEADERS = ["dev_common.h", "formats_dev.h", "group.h", "host_api.h", "host_common.h", "layout.h", "prefill.h"]

HIPCC_FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-Wall",
    # never emit packed fp32 VALU ops (v_pk_*_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc():
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (ROCm is required to build libmoe)")


def build(verbose=False):
    """Compile libmoe.so for gfx950; always recompiles (each source by itself,
    several at a time, then one link)."""
    with tempfile.TemporaryDirectory(prefix="libmoe_") as tmp_dir:
        objects = [os.path.join(tmp_dir, s + ".o") for s in SOURCES]

        def compile_one(job):
            source, obj = job
            return _run([hipcc(), *HIPCC_FLAGS, "-I", os.path.join(ROOT, "include"), "-c",
                         os.path.join(CSRC, source), "-o", obj], verbose)

        with ThreadPoolExecutor(min(len(SOURCES), os.cpu_count() or 1, 8)) as pool:
            list(pool.map(compile_one, zip(SOURCES, objects)))
        tmp = LIB + ".tmp"
        _run([hipcc(), "--offload-arch=gfx950", "-fPIC", "-shared", *objects, "-o", tmp], verbose)
    os.replace(tmp, LIB)
    return LIB


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("hipcc failed building libmoe.so")


if __name__ == "__main__":
    print(build(verbose=True))
