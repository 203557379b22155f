"""Build libspecfold.so in-tree with nvcc for sm_103a (GB300).

Translation units compile in parallel into sparse_reuse_gb300/_build/ and
link into sparse_reuse_gb300/libspecfold.so, for which nvcc is enough.  Where
torch and Python's headers are installed, the CPython module that marshals
torch tensors for the paged-cache calls (PagedCache) is built against it.  A
rebuild is skipped when what there is to build is newer than every source and
header, and the module was built for the installed torch.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libspecfold.so")
TORCH_EXT = os.path.join(PKG, "_sf_torch.so")  # torch argument marshalling of the paged-cache calls
TORCH_STAMP = os.path.join(BUILD, "sf_torch.version")  # the torch it was built for

SOURCES = ["sf_api.cu", "sf_gate.cu", "sf_gemm.cu", "sf_gemm_tc.cu", "sf_attn.cu", "sf_head.cu",
           "sf_cache.cu", "sf_cache_attend.cu", "sf_cache_evict.cu", "sf_cache_rows.cu",
           "sf_cache_rows_tc.cu", "sf_cache_turn.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
                "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecfold")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def _torch_version():
    """The installed torch, which the marshalling module is compiled against; None without torch or Python's headers."""
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return None
    try:
        import torch
    except ImportError:
        return None
    return f"{torch.__version__} {sys.implementation.cache_tag}"


def _built_for():
    try:
        with open(TORCH_STAMP) as f:
            return f.read()
    except OSError:
        return None


def up_to_date() -> bool:
    outputs = [LIB]
    version = _torch_version()
    if version is not None:
        if _built_for() != version:
            return False
        outputs.append(TORCH_EXT)
    if not all(os.path.exists(f) for f in outputs):
        return False
    t = min(os.path.getmtime(f) for f in outputs)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [nvcc()] + FLAGS + list(extra) + ["-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_torch_ext() -> str:
    """Object of the CPython module that marshals torch tensors (host code only)."""
    import torch
    base = os.path.dirname(torch.__file__)
    obj = os.path.join(BUILD, "sf_torch.o")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    incs = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
            sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE]
    for i in incs:
        cmd += ["-isystem", i]
    cmd += ["-c", os.path.join(CSRC, "sf_torch.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for sf_torch.cpp:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link_torch_ext(obj: str) -> None:
    import torch
    tmp = TORCH_EXT + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-L", PKG,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-l:libspecfold.so", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TORCH_EXT)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and not extra and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    version = _torch_version()
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        torch_obj = ex.submit(_compile_torch_ext) if version is not None else None
        objs = list(ex.map(lambda s: _compile(s, extra), srcs))
    tmp = LIB + ".tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if torch_obj is not None:
        _link_torch_ext(torch_obj.result())
        with open(TORCH_STAMP, "w") as f:
            f.write(version)
    if verbose:
        print(f"built {LIB}" + ("" if torch_obj is not None else " (no torch: without PagedCache's marshalling)"),
              file=sys.stderr)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ())
