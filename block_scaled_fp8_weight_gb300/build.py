"""Builds libbsf8.so (the CUDA library behind include/bsf8.h) in-tree for sm_103a.

Each .cu file is compiled to an object in parallel with nvcc, then linked into a shared
library next to this file.  No torch extension machinery is involved: the library is a
plain C-ABI .so that the ctypes binding in __init__.py loads, and neither building nor loading
it needs torch.

csrc/bsf8_torch.cpp, the decode operators' calls from torch tensors, becomes a CPython extension
beside it (g++, torch's headers), built when decode.py first needs it.  Its file name holds the
versions of Python and torch it was compiled against, so that it is not loaded into others.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import threading

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libbsf8.so")
EXT_SOURCE = os.path.join(CSRC, "bsf8_torch.cpp")

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
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")]
    deps.append(os.path.join(INCLUDE, "bsf8.h"))
    deps.append(os.path.abspath(__file__))
    return deps


def _fresh(path, inputs) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in inputs)


def up_to_date() -> bool:
    return _fresh(LIB, _inputs())


def extension_path() -> str:
    """Where the extension for this Python and torch lies."""
    import torch

    torch_tag = "".join(c if c.isalnum() else "_" for c in torch.__version__)
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(HERE, f"_bsf8_torch.{sys.implementation.cache_tag}-torch{torch_tag}-abi{abi}.so")


def _extension_up_to_date() -> bool:
    return _fresh(extension_path(), [EXT_SOURCE, os.path.join(INCLUDE, "bsf8.h"), os.path.abspath(__file__)])


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

    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def _compile_extension() -> str:
    os.makedirs(BUILD, exist_ok=True)
    obj = os.path.join(BUILD, f"bsf8_torch.{os.getpid()}.o")
    cc, _ = _torch_flags()
    r = subprocess.run([*cc, "-c", EXT_SOURCE, "-o", obj], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {EXT_SOURCE}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_extension(obj: str) -> str:
    path = extension_path()
    tmp = path + f".tmp{os.getpid()}"
    _, ld = _torch_flags()
    r = subprocess.run(["g++", "-shared", "-o", tmp, obj, *ld], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking {path} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    os.remove(obj)
    return path


def build_extension(force: bool = False) -> str:
    """Compile the extension for this Python and torch if it is missing or older than its sources (libbsf8.so, which
    it links to, too); return its path."""
    if not os.path.exists(LIB):
        build()
    if not force and _extension_up_to_date():
        return extension_path()
    return _link_extension(_compile_extension())


def build_all(force: bool = False) -> None:
    """The library and the extension, compiled side by side."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_compile_extension) if force or not _extension_up_to_date() else None
        build(force=force)
        if obj is not None:
            _link_extension(obj.result())


_extension = None
_extension_lock = threading.Lock()


def load_extension(build_if_missing: bool = True):
    """The extension as a module (built first if it is missing)."""
    global _extension
    with _extension_lock:
        if _extension is None:
            path = extension_path()
            if not os.path.exists(path):
                if not build_if_missing:
                    raise RuntimeError(f"the decode operators' extension is not built for this torch ({path})")
                build_extension()
            spec = importlib.util.spec_from_file_location(__package__ + "._bsf8_torch", path)
            module = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(module)
            _extension = module
        return _extension


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
