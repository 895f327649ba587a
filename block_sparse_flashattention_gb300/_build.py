"""Compiles the CUDA sources into libbsattn.so (sm_103a) next to this file, and, beside
it, the native form of the cache calls over torch tensors (_torch_calls.so)."""
from __future__ import annotations

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
LIB = os.path.join(PKG, "libbsattn.so")
CALLS = os.path.join(PKG, "_torch_calls.so")
OBJDIR = os.path.join(ROOT, "_build")
CALLS_TORCH = os.path.join(OBJDIR, "torch_calls.version")   # the torch that CALLS was compiled against

NVCC_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def calls_up_to_date(torch_version: str) -> bool:
    """Whether CALLS is newer than its sources and was compiled against this torch."""
    if not os.path.exists(CALLS) or not os.path.exists(CALLS_TORCH):
        return False
    inputs = [os.path.join(CSRC, "torch_calls.cpp"), os.path.join(INCLUDE, "bsattn.h"), os.path.abspath(__file__)]
    with open(CALLS_TORCH) as f:
        return f.read() == torch_version and all(os.path.getmtime(x) <= os.path.getmtime(CALLS) for x in inputs)


def build_calls(force: bool = False) -> bool:
    """Compiles csrc/torch_calls.cpp against the installed torch.  It only spares host time
    (kv_cache.py marshals the same calls through ctypes without it), so that a machine
    where it does not compile goes without: the reason is printed, False returned."""
    src = os.path.join(CSRC, "torch_calls.cpp")
    try:
        import torch
    except ImportError:
        return False
    if not force and calls_up_to_date(torch.__version__):
        return True
    root = os.path.join(os.path.dirname(os.path.abspath(torch.__file__)))
    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.sep in _nvcc() else "/usr/local/cuda"
    tmp = f"{CALLS}.tmp.{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", src, "-o", tmp, "-I" + INCLUDE,
           "-I" + os.path.join(root, "include"), "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"),
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-L" + os.path.join(root, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        print(f"{src} was not compiled, the cache calls go through ctypes:\n{r.stderr}", file=sys.stderr)
        return False
    os.replace(tmp, CALLS)
    os.makedirs(OBJDIR, exist_ok=True)
    with open(CALLS_TORCH, "w") as f:
        f.write(torch.__version__)
    return True


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (in parallel, one translation unit per process) and link."""
    if not force and up_to_date():
        build_calls()
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    nvcc = _nvcc()
    pid = os.getpid()

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src) + f".{pid}.o")
        cmd = [nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            print(r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(sources()) + 1) as ex:
        calls = ex.submit(build_calls, force)
        objs = list(ex.map(compile_one, sources()))
        calls.result()
    tmp = f"{LIB}.tmp.{pid}"
    cmd = [nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    for o in objs:
        os.remove(o)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB
