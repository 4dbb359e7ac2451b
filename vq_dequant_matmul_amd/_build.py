"""Build the HIP library (hipcc, gfx950) in-tree.

The library is one shared object, ``libvqmm.so``, next to this file.  Each
source compiles to an object in ``_build/`` (in parallel), then hipcc links.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libvqmm.so")
SOURCES = ["vq_api.cpp", "vq_decode.hip", "vq_decode_d2.hip", "vq_decode_d4.hip",
           "vq_decode_d8.hip", "vq_prefill.hip", "vq_prefill_d2.hip", "vq_prefill_d4.hip",
           "vq_prefill_d8.hip", "vq_gather.hip", "vq_fit.hip", "vq_probe.hip",
           "vq_block_api.cpp", "vq_q4.hip", "vq_q4_g32.hip", "vq_q4_g64.hip",
           "vq_q4_g128.hip", "vq_route.hip", "vq_norm.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

COMMON = [
    "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    f"--offload-arch={ARCH}",
    # keep the compiler from forming packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unknown-pragmas",
]


def compile_command(src: str, root: str = ROOT) -> list:
    """hipcc's command line for one source of the tree at `root`, without what it makes."""
    package = os.path.basename(HERE)
    return [HIPCC, "-x", "hip", *COMMON, "-I", os.path.join(root, "include"),
            os.path.join(root, package, "csrc", src)]


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    r = subprocess.run([*compile_command(src), *extra, "-c", "-o", obj], capture_output=True,
                       text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def build(extra=(), jobs: int = 8, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    # a build that fails leaves no library, and no object that another link could take
    for old in [LIB] + [os.path.join(BUILD, os.path.splitext(s)[0] + ".o") for s in SOURCES]:
        if os.path.exists(old):
            os.remove(old)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, list(extra)), SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
