"""Build the gfx950 HIP library libfftconv.so in-tree with hipcc.

Run ``python -m long_fft_convolution_amd.build`` (or ``__graft_entry__.build()``).
Every HIP source is compiled for gfx950 only, with packed-fp32 instruction
selection disabled; the objects are linked into one shared library next to
this file.
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libfftconv.so")
BUILD_DIR = os.path.join(HERE, "_build")

SOURCES = ["delta_f32.hip", "delta_bf16.hip", "delta_f16.hip", "multipass.hip", "pair16k.hip", "pair_mfma.hip", "decay_f32.hip", "decay_bf16.hip", "decay_f16.hip",
           "linear_bf16.hip", "linear_f16.hip", "linear_f32.hip", "fused.hip", "eqlinear.hip", "bwd.hip", "filter.hip",
           "norm.hip", "api.cpp", "sequence_ops.cpp", "norm_ops.cpp", "delta_ops.cpp"]   # the longest compilations first

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I" + os.path.join(HERE, "..", "include"),
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-x", "hip", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stderr}")
    return obj


def build(verbose: bool = True) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = OUT + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, OUT)
    if verbose:
        print(f"built {OUT}", file=sys.stderr)
    return OUT


if __name__ == "__main__":
    build()
