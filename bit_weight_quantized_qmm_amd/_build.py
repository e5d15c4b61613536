"""Build libqmm.so (the C-ABI library) for gfx950 with hipcc, in-tree, and
_binding.so, the CPython side of the decoder-layer calls.

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
BINDING = os.path.join(PKG, "_binding.so")
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


def build_binding() -> str:
    """_binding.so: the CPython side of the decoder-layer calls, against torch's C++ headers (host code only)."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    inc = cpp_extension.include_paths() + [sysconfig.get_paths()["include"]]
    libs = cpp_extension.library_paths()
    tmp = BINDING + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-w", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    cmd += [f"-isystem{p}" for p in inc] + [os.path.join(CSRC, "binding.cpp"), "-o", tmp]
    cmd += [f"-L{p}" for p in libs] + ["-ltorch_python", "-ltorch_cpu", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{res.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


def build(jobs: int = 8) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(jobs, len(SOURCES))) as ex:
        binding = ex.submit(build_binding)
        objs = list(ex.map(_compile, SOURCES))
        binding.result()
    tmp = LIBRARY + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stderr}")
    os.replace(tmp, LIBRARY)
    return LIBRARY


if __name__ == "__main__":
    print(build())
