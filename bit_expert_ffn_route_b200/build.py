"""Build libmoe.so (the CUDA library behind include/moe.h) for sm_100a, and the
native binding of moe_ops.h (_ops.so, a Python extension module), in-tree.

    python -m bit_expert_ffn_route_b200.build [--force]

nvcc cross-compiles here without a GPU; the .so lands next to this file.  The
extension module needs a C++ compiler and torch's headers: without them the build
warns, and moe.py raises at the first use of one of its calls.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libmoe.so")
OPS_SRC, OPS = os.path.join(CSRC, "binding.cpp"), os.path.join(HERE, "_ops.so")
OPS_FOR = os.path.join(BUILD, "_ops.for")       # the versions of torch and Python that it was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _read(path):
    if not os.path.exists(path):
        return None
    with open(path) as f:
        return f.read()


def _ops_command():
    import sysconfig

    import torch
    at = os.path.dirname(torch.__file__)
    include = [os.path.join(at, "include"), os.path.join(at, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
            f'-DMOE_TORCH_VERSION="{torch.__version__}"', "-I", INCLUDE,
            *(f"-isystem{i}" for i in include), OPS_SRC, "-o", OPS, "-L" + os.path.join(at, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda", "-L" + HERE, "-l:libmoe.so", "-Wl,-rpath,$ORIGIN"]


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    headers = _headers()
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            jobs.append([NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj] + (["-Xptxas", "-v"] if verbose else []))

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        return r.stderr

    with ThreadPoolExecutor(max_workers=max(1, os.cpu_count() or 1)) as ex:
        for out in ex.map(run, jobs):
            if verbose and out:
                sys.stderr.write(out)
    if force or jobs or _stale(LIB, objs):
        subprocess.run([NVCC, *ARCH, "-shared", "-o", LIB, *objs, "-lcudart"], check=True)
    try:
        import torch
        versions = f"torch {torch.__version__}, Python {sys.version_info[0]}.{sys.version_info[1]}"
        if force or _stale(OPS, [OPS_SRC, LIB] + headers) or _read(OPS_FOR) != versions:
            if os.path.exists(OPS):             # of other sources, or for another torch: not to be loaded
                os.remove(OPS)
            run(_ops_command())
            with open(OPS_FOR, "w") as f:
                f.write(versions)
    except (RuntimeError, OSError, ImportError) as e:           # the compiler's errors, no compiler, no torch
        warnings.warn(f"{OPS} was not built: the calls of moe_ops.h cannot be used from Python ({e})", RuntimeWarning)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
