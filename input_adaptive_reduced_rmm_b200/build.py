"""Build librmm.so in-tree: nvcc for sm_100a, one object per .cu, then a shared link;
and _binding.so, the Python module in front of some of its calls (g++, against torch).

    python -m input_adaptive_reduced_rmm_b200.build [--force] [--verbose-ptxas]

The library links the CUDA runtime statically and reaches the driver API
(tensor-map encoding) through cudaGetDriverEntryPoint, so it loads on a
machine without a GPU (only calls into it need one).
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "librmm.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
BINDING_FOR = os.path.join(OBJ, "_binding.for")  # what it was compiled against

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Werror", "all-warnings", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _deps():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu*")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, verbose_ptxas):
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    if not _stale(obj, [src] + headers):
        return obj, ""
    cmd = [NVCC] + ARCH + CFLAGS + (["-Xptxas", "-v"] if verbose_ptxas else []) + ["-c", src, "-o", obj]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{p.stdout}\n{p.stderr}")
    return obj, p.stderr


def _binding_target():
    """The torch and Python that the module uses the C++ and C interfaces of: it fits no others."""
    import torch

    return f"torch {torch.__version__} {torch.version.git_version} {torch.compiled_with_cxx11_abi()}, " \
           f"python {sys.implementation.cache_tag} {sys.hexversion:#x}\n"


def _binding_stale():
    if _stale(BINDING, [BINDING_SRC, os.path.join(INCLUDE, "rmm.h")]):
        return True
    try:
        with open(BINDING_FOR) as f:
            return f.read() != _binding_target()
    except OSError:
        return True


def _build_binding(force):
    """Compile csrc/binding.cpp into _binding.so, which finds librmm.so beside itself."""
    if not force and not _binding_stale():
        return
    import torch
    from torch.utils import cpp_extension

    inc = cpp_extension.include_paths() + [INCLUDE, sysconfig.get_paths()["include"],
                                           os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    libs = [os.path.join(os.path.dirname(torch.__file__), "lib")]
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = (["g++", "-O2", "-std=c++17", "-shared", "-fPIC", BINDING_SRC, "-o", tmp] + [f"-I{i}" for i in inc] +
           [f"-L{p}" for p in libs] + [f"-L{PKG}", "-l:librmm.so", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
                                       "-lc10_cuda", "-Wl,-rpath,$ORIGIN"])
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"g++ failed for {BINDING_SRC}:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_FOR + f".tmp{os.getpid()}", "w") as f:
        f.write(_binding_target())
    os.replace(BINDING_FOR + f".tmp{os.getpid()}", BINDING_FOR)


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile every csrc/*.cu for sm_100a and link librmm.so, then the Python module;
    returns the library's path."""
    _build_library(force, verbose_ptxas)
    _build_binding(force)
    return LIB


def _build_library(force, verbose_ptxas):
    os.makedirs(OBJ, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    if not force and not verbose_ptxas and not _stale(LIB, _deps()):
        return
    if force:
        for o in glob.glob(os.path.join(OBJ, "*.o")):
            os.remove(o)
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose_ptxas), srcs))
    if verbose_ptxas:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", tmp] + objs
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose_ptxas=a.verbose_ptxas))
