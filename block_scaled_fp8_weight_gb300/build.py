"""Builds libbsf8.so (the CUDA library behind include/bsf8.h) in-tree for sm_103a.

Each .cu file is compiled to an object in parallel with nvcc, then linked into a shared
library next to this file.  No torch extension machinery is involved: the library is a
plain C-ABI .so that the ctypes binding in __init__.py loads.  csrc/bsf8_torch.cpp, the
decode operators' calls from torch tensors, becomes a CPython extension beside it (g++,
torch's headers).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libbsf8.so")
EXT = os.path.join(HERE, "_bsf8_torch.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libbsf8")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _inputs():
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    deps.append(os.path.join(INCLUDE, "bsf8.h"))
    deps.append(os.path.abspath(__file__))
    return deps


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(EXT):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
    return all(os.path.getmtime(d) <= t for d in _inputs())


def _torch_flags():
    """Compile and link flags of the extension: torch's and Python's headers, torch's libraries."""
    import sysconfig

    import torch

    root = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), INCLUDE]
    cc = ["g++", "-O2", "-std=c++17", "-fPIC", *[f"-I{i}" for i in inc],
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    ld = [f"-L{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", f"-L{HERE}",
          "-l:libbsf8.so", "-Wl,-rpath,$ORIGIN"]
    return cc, ld


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile libbsf8.so if it is missing or older than its sources; return its path."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if ptxas_info or verbose:
            sys.stderr.write(r.stderr)
        return obj

    ext_obj = os.path.join(BUILD, "bsf8_torch.o")
    ext_cc, ext_ld = _torch_flags()

    def compile_ext():
        cmd = [*ext_cc, "-c", os.path.join(CSRC, "bsf8_torch.cpp"), "-o", ext_obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for bsf8_torch.cpp:\n{r.stdout}\n{r.stderr}")

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        ext = ex.submit(compile_ext)
        objs = list(ex.map(compile_one, srcs))
        ext.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    tmp = EXT + f".tmp{os.getpid()}"
    r = subprocess.run(["g++", "-shared", "-o", tmp, ext_obj, *ext_ld], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {EXT} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
