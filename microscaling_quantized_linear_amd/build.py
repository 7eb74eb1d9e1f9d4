"""Build libmx.so (the HIP kernels and the C ABI of include/mx.h) for gfx950.

    python -m microscaling_quantized_linear_amd.build

Objects go to ``_build/`` next to this file; the library is written in-tree as
``microscaling_quantized_linear_amd/libmx.so``, the binding's compiled call path
as ``_mxcall`` (with this Python's extension suffix) next to it.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmx.so")
CALL = os.path.join(HERE, "_mxcall" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["mx_pack.hip", "mx_ingest.hip", "mx_quant.hip", "mx_gemv.hip", "mx_gemv_w8.hip",
           "mx_gemm.hip", "mx_static.hip", "mx_norm.hip", "mx_route.hip", "mx_grouped.hip",
           "mx_grouped_gemm.hip", "mx_lora.hip", "mx_gemv_epi.hip", "mx_gemv_w8_epi.hip",
           "mx_gemm_epi.hip", "mx_router.hip", "mx_block.hip", "mx_plan.cpp", "mx_api.cpp", "mx_ops_api.cpp",
           "mx_layer_api.cpp"]

HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # packed fp32 ops off: see the note on v_pk_* in the design notes
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function", "-Wno-unused-variable",
]


def _compile(src: str) -> str:
    obj = os.path.join(OUT, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".cpp"):
        cmd = [HIPCC, "-O2", "-std=c++17", "-fPIC", "-Wall", "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compile of {src} failed:\n{r.stdout}\n{r.stderr}")
    return obj


def build_call() -> str:
    """The binding's call path (csrc/mx_python.cpp): host code against Python's headers.
    It is imported ahead of torch, so it must not bring in the HIP runtime (hipcc links
    it): torch loads its own, and two of them in a process do not share a device."""
    tmp = CALL + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-shared",
           "-I" + sysconfig.get_paths()["include"], os.path.join(CSRC, "mx_python.cpp"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"build of mx_python.cpp failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL)
    return CALL


def build(verbose: bool = False) -> str:
    os.makedirs(OUT, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(SOURCES))) as ex:
        call = ex.submit(build_call)
        objs = list(ex.map(_compile, SOURCES))
        call.result()
    tmp = LIB + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
