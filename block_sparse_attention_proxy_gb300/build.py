"""Builds libmsa.so in-tree with nvcc for sm_103a (GB300), and the torch front end of the
dense attention (_dense_torch.so, host C++) that calls it.

Each CUDA source compiles to its own object in parallel under ``_build/``;
objects newer than every source and header are reused.  The CUDA runtime is
linked statically and the driver entry point for tensor maps is resolved at run
time, so the library loads on machines without a GPU driver (its entry points
then fail with MSA_ERR_CUDA).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmsa.so")
TORCH_LIB = os.path.join(PKG, "_dense_torch.so")
INCLUDE = os.path.join(ROOT, "include")

SOURCES = ["msa_api.cu", "k_regroup.cu", "k_select.cu", "k_selarg.cu", "k_fwd.cu", "k_bwd.cu",
           "k_reduce.cu", "msa_noalloc.cu", "k_dense_fwd.cu", "k_dense_bwd.cu", "msa_dense.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libmsa")
    return path


def _deps() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "msa.h")]
    return max(os.path.getmtime(f) for f in files)


def _compile(src: str, newest: float, extra: list[str]) -> str:
    obj = os.path.join(BUILD, src.replace(".cu", ".o"))
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_torch(newest: float) -> str:
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    obj, stamp = (os.path.join(BUILD, "dense_torch" + x) for x in (".o", ".stamp"))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    dirs = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"],
            os.path.join(cuda, "include")]
    cmd = ["g++", "-O1", "-std=c++17", "-fPIC", "-DTORCH_EXTENSION_NAME=_dense_torch",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           *(x for d in dirs for x in ("-isystem", d)), "-c",
           os.path.join(CSRC, "dense_torch.cpp"), "-o", obj]
    # the object is tied to the C++ interface of this torch and this Python
    made_for = "\n".join([torch.__version__, str(sysconfig.get_config_var("SOABI")), *cmd])
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == made_for:
                return obj
    if os.path.exists(stamp):
        os.remove(stamp)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for dense_torch.cpp:\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(made_for)
    return obj


def _link_torch(obj: str) -> None:
    from torch.utils import cpp_extension

    if os.path.exists(TORCH_LIB) and os.path.getmtime(TORCH_LIB) >= os.path.getmtime(obj):
        return
    libs = [x for d in cpp_extension.library_paths() for x in ("-L", d)]
    tmp = TORCH_LIB + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, *libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch",
           "-ltorch_python", "-L", PKG, "-l:libmsa.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_LIB)


def build(verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile (if needed) and return the path of libmsa.so."""
    os.makedirs(BUILD, exist_ok=True)
    newest = _deps()
    extra = list(extra_flags or [])
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        front = ex.submit(_compile_torch, newest)
        objs = list(ex.map(lambda s: _compile(s, newest, extra), SOURCES))
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + ".tmp"
        cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _link_torch(front.result())
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
