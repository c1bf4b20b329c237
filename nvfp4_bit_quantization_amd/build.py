"""Build libnvfp4.so (the HIP kernels and the C ABI) in-tree with hipcc for gfx950.

    python -m nvfp4_bit_quantization_amd.build

Compiles every translation unit under csrc/ in parallel into _build/ and links
nvfp4_bit_quantization_amd/libnvfp4.so.  Always recompiles (the build check
runs it every time); the Python binding loads the library and never builds.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libnvfp4.so")
SOURCES = ["quantize.hip", "gemm.hip", "mxfp4.hip", "api.cpp", "norm.hip", "adamw.hip", "attention.hip", "train_api.cpp",
           "rope.hip", "gated.hip", "muon.hip", "block_api.cpp"]
ARCH = "gfx950"

FLAGS = [
    "-O3", "-std=c++17", "--offload-arch=" + ARCH, "-fPIC",
    # the scale chain is single binary32 operations: no FMA contraction, IEEE
    # division, denormals kept
    "-ffp-contract=off", "-fno-gpu-flush-denormals-to-zero", "-fhip-fp32-correctly-rounded-divide-sqrt",
    # packed-FP32 instructions disabled on this platform
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", os.path.join(ROOT, "include"), "-I", CSRC,
]

# attention: no NaN arises from finite inputs that keep scores finite, and maxima
# need no quieting
FILE_FLAGS = {"attention.hip": ["-fno-honor-nans"]}


def hipcc() -> str:
    for c in (shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("hipcc not found")


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, src + ".o")
    cmd = [hipcc()] + FLAGS + FILE_FLAGS.get(src, []) + ["-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s" % (src, r.stderr[-6000:]))
    return obj


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    jobs = min(len(SOURCES), max(1, int(os.environ.get("MAX_JOBS", "8"))))
    with ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [hipcc(), "--offload-arch=" + ARCH, "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stderr[-4000:])
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
