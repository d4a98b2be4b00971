"""Build libgdn.so (the C ABI declared in include/gdn.h) for sm_103a with nvcc.

Each .cu translation unit compiles in parallel to an object file under
``_build/``; the objects link into ``libgdn.so`` next to this file (in-tree,
never installed). The binding's extension (``binding_ext.cpp``, the host compiler,
PyTorch's headers) compiles beside them and links against it. Only one ``-gencode``
(compute_103a -> sm_103a) is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sysconfig
from typing import List, Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libgdn.so")
EXT_PATH = os.path.join(PKG, "_gdn_ext.so")  # the binding's compiled argument marshalling
SOURCES = ["api.cu", "recurrent.cu", "decode.cu", "l2norm.cu", "chunk_fwd.cu", "chunk_bwd.cu",
           "chunk_grads.cu", "chunk_scan_tc.cu", "chunk_bwd_tc.cu", "chunk_prep_tc.cu", "chunk_merge.cu", "noalloc.cu", "replay.cu",
           "api_hybrid.cu", "block_norm.cu", "kv_append.cu", "paged_attn.cu", "paged_attn_tc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc_path() -> str:
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the gated delta rule library needs the CUDA toolkit to build")
    return cand


def _inputs() -> List[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    files.append(os.path.join(INCLUDE, "gdn.h"))
    files.append(os.path.abspath(__file__))
    return files


def is_stale() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(EXT_PATH):
        return True
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(EXT_PATH))
    return any(os.path.getmtime(f) > t for f in _inputs())


def ext_commands(out: str) -> List[List[str]]:
    """Compile and link commands of the binding's extension (PyTorch's headers and libraries)."""
    import torch

    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc_path()))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    obj = os.path.join(BUILD_DIR, "binding_ext.o")
    cxx = os.environ.get("CXX", "g++")
    return [[cxx, "-O2", "-std=c++17", "-fPIC", *(f"-I{i}" for i in inc),
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             "-c", os.path.join(CSRC, "binding_ext.cpp"), "-o", obj],
            [cxx, "-shared", "-o", out, obj, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
             "-lc10_cuda", "-L" + PKG, "-l:libgdn.so", "-Wl,-rpath,$ORIGIN"]]


def _run(what: str, cmd: List[str], verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout, r.stderr, flush=True)


def build(force: bool = False, verbose: bool = False, extra_flags: Optional[List[str]] = None) -> str:
    """Compile and link libgdn.so and the binding's extension if missing or older than their sources."""
    if not force and not is_stale():
        return LIB_PATH
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        _run(f"nvcc on {src}", [nvcc, *flags, "-c", os.path.join(CSRC, src), "-o", obj], verbose)
        return obj

    tmp, ext_tmp = (f"{p}.{os.getpid()}.tmp" for p in (LIB_PATH, EXT_PATH))
    ext_compile, ext_link = ext_commands(ext_tmp)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        ext = ex.submit(_run, "compiling binding_ext.cpp", ext_compile, verbose)
        objs = list(ex.map(compile_one, SOURCES))
        ext.result()
    _run("link", [nvcc, *ARCH, "-shared", "-o", tmp, *objs], verbose)
    os.replace(tmp, LIB_PATH)
    _run("link of the binding's extension", ext_link, verbose)
    os.replace(ext_tmp, EXT_PATH)
    return LIB_PATH


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose=True))
