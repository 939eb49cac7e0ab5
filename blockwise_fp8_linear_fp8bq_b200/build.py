"""Build libfp8bq.so (the C-ABI CUDA library) in-tree with nvcc for sm_100a, and
_row_binding.so (the compiled Python binding of the row operators) with g++.

    python -m blockwise_fp8_linear_fp8bq_b200.build [--force] [--verbose]

IEEE arithmetic is kept (no --use_fast_math, no -ftz): the quantizers must be
bit-exact and scales may be fp32 subnormals.
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libfp8bq.so")
BINDING_SRC = os.path.join(CSRC, "row_binding.cpp")
BINDING = os.path.join(HERE, "_row_binding.so")
BINDING_TORCH = os.path.join(BUILD, "row_binding.torch")  # the torch that the binding was built against

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found")
    return path


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h")))


def _older(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def needs_build() -> bool:
    return _older(LIB, _deps()) or needs_binding()


def torch_version() -> str:
    import torch
    return torch.__version__


def needs_binding() -> bool:
    """Whether the binding is missing, older than its sources, or another torch's."""
    if _older(BINDING, [BINDING_SRC] + glob.glob(os.path.join(INCLUDE, "*.h"))):
        return True
    try:
        with open(BINDING_TORCH) as f:
            return f.read() != torch_version()
    except FileNotFoundError:
        return True


def build_binding(verbose: bool = False) -> str:
    """_row_binding.so, against the headers and libraries of the installed torch."""
    import torch
    from torch.utils import cpp_extension

    cuda = os.path.dirname(os.path.dirname(nvcc()))
    includes = [INCLUDE, *cpp_extension.include_paths(), sysconfig.get_path("include"), os.path.join(cuda, "include")]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    version = torch_version()
    cmd = ["g++", f'-DFP8BQ_TORCH_VERSION="{version}"', "-O2", "-std=c++17", "-shared", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[a for i in includes for a in ("-isystem" if i != INCLUDE else "-I", i)], BINDING_SRC, "-o", tmp,
           f"-L{libs}", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-lc10", "-lc10_cuda", "-ldl"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0 or verbose:
        sys.stderr.write(r.stderr)
    if r.returncode != 0:
        raise RuntimeError("g++ failed on row_binding.cpp")
    os.replace(tmp, BINDING)
    os.makedirs(BUILD, exist_ok=True)
    with open(BINDING_TORCH, "w") as f:
        f.write(version)
    return BINDING


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    if not force and not needs_build():
        return LIB
    if not force and not _older(LIB, _deps()):
        build_binding(verbose)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        return src, obj, subprocess.run(cmd, capture_output=True, text=True)

    objs = []
    with ThreadPoolExecutor(os.cpu_count() or 1) as pool:
        binding = pool.submit(build_binding, verbose) if force or needs_binding() else None
        for src, obj, r in pool.map(compile_one, _sources()):
            if r.returncode != 0 or ((verbose or ptxas_info) and r.stderr):
                sys.stderr.write(r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {os.path.basename(src)}")
            objs.append(obj)
        if binding is not None:
            binding.result()
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    ap.add_argument("--ptxas-info", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force or a.ptxas_info, verbose=a.verbose, ptxas_info=a.ptxas_info))
