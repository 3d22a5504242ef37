"""Build libmoe2bit.so (HIP kernels + C ABI) in-tree for gfx950 with hipcc.

Every source is compiled on each call; object files go to _build/ next to this
file and the shared library to libmoe2bit.so.  hipcc cross-compiles, so no GPU
is needed.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe2bit.so")
SOURCES = ["api.cpp", "prep.hip", "route.hip", "ffn_generic.hip", "ffn_gemv.hip", "ffn_gemm.hip", "combine.hip", "norm.hip",
           "ffn_shared.hip", "grouped.hip", "q4_32.hip", "q4_64.hip", "q4_128.hip", "probe.hip"]

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
    # a host function that runs off its end goes on in other code; a packed struct that is not packed promises an alignment
    "-Werror=return-type", "-Werror=packed-non-pod",
    # no packed-fp32 code generation (v_pk_*_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, src + ".o")
    cmd = [HIPCC, *FLAGS, "-I", os.path.join(HERE, "..", "include"), "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd[1:1] = ["-x", "hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    # (the host side does not know the target feature, and says how often it said so)
    errs = "\n".join(l for l in r.stderr.splitlines()
                     if "packed-fp32-ops" not in l and "unknown target feature" not in l
                     and not l.endswith(("warning generated when compiling for host.", "warnings generated when compiling for host.")))
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{errs}")
    if errs.strip():
        print(f"{src}:\n{errs}", file=sys.stderr, flush=True)
    return obj


def build(jobs: int = 8) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    subprocess.check_call([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build())
    sys.exit(0)
