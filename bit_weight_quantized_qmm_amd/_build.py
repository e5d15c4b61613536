"""Build libqmm.so (the C-ABI library) for gfx950 with hipcc, in-tree.

Every translation unit is compiled to an object under ``_build/`` in parallel,
then linked into ``bit_weight_quantized_qmm_amd/libqmm.so``.  All HIP code is
compiled with packed-fp32 instructions disabled (hipcc's host pass warns that
it does not know that feature; the warning is harmless).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build")
LIBRARY = os.path.join(PKG, "libqmm.so")
# (source, object suffix, defines): the product kernels are compiled once without and once with an epilogue
EPILOGUE = ["-DQMM_EPILOGUE"]
SOURCES = [("gemv.hip", "", []), ("gemv.hip", ".linear", EPILOGUE), ("gemm.hip", "", []), ("gemm.hip", ".linear", EPILOGUE),
           ("w4a8.hip", "", []), ("stream.hip", "", []), ("abi.cpp", "", []), ("pack.hip", "", []), ("quantize.hip", "", []), ("probe.hip", "", []),
           ("lut.hip", "", []), ("append.hip", "", []), ("attend.hip", "", [])]
ARCH = "gfx950"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-I", os.path.join(ROOT, "include")]


def _compile(item) -> str:
    src, suffix, defines = item
    obj = os.path.join(BUILD_DIR, src + suffix + ".o")
    cmd = [HIPCC] + COMMON + DEVICE_FLAGS + defines + ["-c", os.path.join(CSRC, src), "-o", obj]
    if src.endswith(".hip"):
        cmd[1:1] = ["-x", "hip"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{res.stderr}")
    return obj


def build(jobs: int = 8) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(jobs, len(SOURCES))) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIBRARY + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIBRARY)
    return LIBRARY


if __name__ == "__main__":
    print(build())
