"""Build libsage.so (the C-ABI library) in-tree with nvcc for sm_100a, and
_serving.so (the Python side of the serving calls) with g++.

    python -m quantized_attention_08_b200.build [--verbose]
"""
from __future__ import annotations

import concurrent.futures
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libsage.so")
SERVING = os.path.join(PKG, "_serving.so")
SERVING_SOURCE = os.path.join(CSRC, "serving_binding.cpp")
SOURCES = ["prepass.cu", "attn_sm100.cu", "kvcache.cu", "rope_axes.cu", "attn_decode.cu", "sage_api.cu"]
HEADERS = ["sage_ptx.cuh", "sage_internal.h", "serve_internal.h", "serve_math.cuh", "quant_div.h", "quant_pair.cuh"]
NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _inputs():
    files = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    files.append(os.path.join(ROOT, "include", "sage.h"))
    return files


def _older(target: str, files) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(f) > t for f in files)


def is_stale() -> bool:
    return _older(LIB, _inputs())


def _run(cmd, target: str, what: str, verbose: bool):
    """Run a compiler whose output is `target`.  It appears whole or not at all, also
    if another process builds it at the same time."""
    tmp = f"{target}.{os.getpid()}.tmp"
    try:
        res = subprocess.run([*cmd, "-o", tmp], capture_output=True, text=True)
        if verbose or res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
        if res.returncode != 0:
            raise RuntimeError(f"building {what} failed:\n" + res.stderr[-4000:])
        os.replace(tmp, target)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)


def _objects(force: bool, verbose: bool):
    """Every CUDA source compiled to an object file, a process a source."""
    os.makedirs(OBJ, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in HEADERS] + [os.path.join(ROOT, "include", "sage.h")]
    objects = [os.path.join(OBJ, s + ".o") for s in SOURCES]
    with concurrent.futures.ThreadPoolExecutor(len(SOURCES)) as pool:
        jobs = []
        for source, obj in zip(SOURCES, objects):
            path = os.path.join(CSRC, source)
            if not force and not _older(obj, [path, *headers]):
                continue
            cmd = [_nvcc(), *NVCC_FLAGS, "-I", os.path.join(ROOT, "include"),
                   *(["-Xptxas", "-v"] if verbose else []), "-c", path]
            jobs.append(pool.submit(_run, cmd, obj, source, verbose))
        for j in jobs:
            j.result()
    return objects


def build_serving(verbose: bool = False, force: bool = False) -> str:
    """Compile the Python side of the serving calls next to this file."""
    header = os.path.join(ROOT, "include", "sage.h")
    if not force and not _older(SERVING, [SERVING_SOURCE, header]):
        return SERVING
    import torch
    at = os.path.join(os.path.dirname(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda"
    include = [os.path.join(ROOT, "include"), os.path.join(at, "include"),
               os.path.join(at, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include"),
               sysconfig.get_paths()["include"]]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *[x for i in include for x in ("-I", i)], SERVING_SOURCE, "-L", os.path.join(at, "lib"),
          "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"], SERVING, "_serving.so", verbose)
    return SERVING


def build(verbose: bool = False, force: bool = False) -> str:
    """Compile every CUDA source into libsage.so next to this file, and the
    serving calls' Python side."""
    if force or is_stale():
        _run([_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", *_objects(force, verbose)],
             LIB, "libsage.so", verbose)
    build_serving(verbose, force)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
