"""Build the HIP library in-tree: paged_layout_transfer_amd/libkvxfer.so (gfx950 only)."""
from __future__ import annotations

import os
import subprocess
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libkvxfer.so")
# the transfer path, then the operators on the cache beside it
SOURCES = [os.path.join(CSRC, "kvxfer.cpp"), os.path.join(CSRC, "kvxfer_kernels.hip")]
OPERATORS = [os.path.join(CSRC, f) for f in ("kvxfer_ops.cpp", "kvxfer_pages.hip", "kvxfer_attn_f16.hip",
                                             "kvxfer_attn_bf16.hip")]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared",
    "-fvisibility=hidden",
    # no packed-fp32 instructions anywhere in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-command-line-argument",
]


def build_library(force: bool = True) -> str:
    """Compiles every source (side by side) and links the library."""
    if not force and os.path.exists(LIB):
        return LIB
    objects = os.path.join(HERE, "build")
    os.makedirs(objects, exist_ok=True)

    def run(cmd):
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("hipcc failed:\n" + res.stdout + res.stderr)

    def compile_one(src):
        obj = os.path.join(objects, os.path.basename(src) + ".o")
        run([HIPCC, *[f for f in FLAGS if f != "-shared"], "-I", os.path.join(ROOT, "include"), "-I", CSRC,
             "-c", src, "-o", obj])
        return obj

    with ThreadPoolExecutor(max_workers=4) as pool:
        objs = list(pool.map(compile_one, SOURCES + OPERATORS))
    tmp = LIB + ".tmp"
    run([HIPCC, "--offload-arch=gfx950", "-fPIC", "-shared", *objs, "-o", tmp])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build_library())
