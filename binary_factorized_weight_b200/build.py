"""Build libdbf.so (the C ABI of include/dbf.h) in-tree with nvcc for sm_100a.

    python -m binary_factorized_weight_b200.build [--force] [-v]

The shared library is written next to this file so that it travels with the
repository; nothing is installed into site-packages.  Compilation is one nvcc
call per .cu file (in parallel) followed by one link.  Beside it goes
_mx_binding.so, the C++ part of the Python binding (csrc/binding.cpp), compiled
with g++ against the installed torch's headers.
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libdbf.so")
BINDING = os.path.join(HERE, "_mx_binding.so")
BUILD_DIR = os.path.join(ROOT, "_build")

SOURCES = ["dbf_api.cu", "decode.cu", "fused.cu", "prefill.cu", "pack.cu", "transpose.cu", "reconstruct.cu", "bqq.cu", "factorize.cu", "noalloc.cu",
           "mx_quantize.cu", "mx_forward.cu", "rmsnorm.cu"]
HEADERS = ["dbf_device.cuh", "mx_device.cuh", "dbf_internal.h"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "--expt-relaxed-constexpr",
    "-I", INCLUDE,
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _fingerprint() -> str:
    h = hashlib.sha256()
    for name in SOURCES + HEADERS:
        with open(os.path.join(CSRC, name), "rb") as f:
            h.update(name.encode() + f.read())
    with open(os.path.join(INCLUDE, "dbf.h"), "rb") as f:
        h.update(f.read())
    h.update(" ".join(NVCC_FLAGS).encode())
    return h.hexdigest()


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile _mx_binding.so for the torch that is installed."""
    import torch

    src = os.path.join(CSRC, "binding.cpp")
    h = hashlib.sha256(f"{torch.__version__} {sys.version}".encode())
    for name in (src, os.path.join(INCLUDE, "dbf.h")):
        with open(name, "rb") as f:
            h.update(f.read())
    stamp, fp = BINDING + ".stamp", h.hexdigest()
    if not force and os.path.exists(BINDING) and os.path.exists(stamp) and open(stamp).read() == fp:
        return BINDING
    from torch.utils import cpp_extension

    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    tmp = BINDING + f".tmp{os.getpid()}"
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-I{p}" for p in cpp_extension.include_paths()], f"-I{sysconfig.get_paths()['include']}",
           f"-I{os.path.join(cuda, 'include')}", src, "-o", tmp, f"-L{lib}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{res.stdout}\n{res.stderr}")
    if verbose:
        sys.stderr.write(res.stdout + res.stderr)
    os.replace(tmp, BINDING)
    with open(stamp, "w") as f:
        f.write(fp)
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    build_binding(force=force, verbose=verbose)
    stamp = LIB + ".stamp"
    fp = _fingerprint()
    if not force and os.path.exists(LIB) and os.path.exists(stamp) and open(stamp).read() == fp:
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(res.stdout + res.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as pool:
        objs = list(pool.map(compile_one, SOURCES))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-Xcompiler", "-fPIC", "-o", tmp, *objs,
           "-lcublas", "-lcusolver"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    with open(stamp, "w") as f:
        f.write(fp)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv))
