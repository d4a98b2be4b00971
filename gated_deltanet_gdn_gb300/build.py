"""Build libgdn.so (the C ABI declared in include/gdn.h) for sm_103a with nvcc.

Each .cu translation unit compiles in parallel to an object file under
``_build/``; the objects link into ``libgdn.so`` next to this file (in-tree,
never installed). The binding's extension (``binding_ext.cpp``, the host compiler,
PyTorch's headers) compiles beside them and links against it; the library does not need it.
Only one ``-gencode`` (compute_103a -> sm_103a) is built.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
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


def _older(path: str, suffixes) -> bool:
    """Whether `path` is missing, or older than the sources with these suffixes, the header or this file."""
    if not os.path.exists(path):
        return True
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(suffixes)]
    t = os.path.getmtime(path)
    return any(os.path.getmtime(f) > t for f in files + [os.path.join(INCLUDE, "gdn.h"), os.path.abspath(__file__)])


def lib_is_stale() -> bool:
    return _older(LIB_PATH, (".cu", ".cuh", ".h"))


def _ext_stamp() -> str:
    return os.path.join(BUILD_DIR, "binding_ext.stamp")


def _ext_against() -> str:
    """What the extension's binary interface depends on beside its source."""
    import torch

    return f"Python {sys.version}, PyTorch {torch.__version__}"


def ext_is_stale() -> bool:
    """Also when it was compiled against another Python or PyTorch."""
    if _older(EXT_PATH, (".cpp",)) or not os.path.exists(_ext_stamp()):
        return True
    with open(_ext_stamp()) as f:
        return f.read() != _ext_against()


def is_stale() -> bool:
    return lib_is_stale() or ext_is_stale()


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


def build_lib(force: bool = False, verbose: bool = False, extra_flags: Optional[List[str]] = None) -> str:
    """Compile and link libgdn.so if missing or older than its sources."""
    if not force and not lib_is_stale():
        return LIB_PATH
    nvcc = nvcc_path()
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = NVCC_FLAGS + list(extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        _run(f"nvcc on {src}", [nvcc, *flags, "-c", os.path.join(CSRC, src), "-o", obj], verbose)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = f"{LIB_PATH}.{os.getpid()}.tmp"
    _run("link", [nvcc, *ARCH, "-shared", "-o", tmp, *objs], verbose)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def _compile_ext(verbose: bool) -> List[str]:
    """Compile the binding's extension; its link command."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    compile_, link = ext_commands(f"{EXT_PATH}.{os.getpid()}.tmp")
    _run("compiling binding_ext.cpp", compile_, verbose)
    return link


def _link_ext(link: List[str], verbose: bool) -> str:
    _run("link of the binding's extension", link, verbose)
    os.replace(link[link.index("-o") + 1], EXT_PATH)
    with open(_ext_stamp(), "w") as f:
        f.write(_ext_against())
    return EXT_PATH


def build_ext(verbose: bool = False) -> str:
    """Compile the binding's extension and link it against libgdn.so."""
    return _link_ext(_compile_ext(verbose), verbose)


def build(force: bool = False, verbose: bool = False, extra_flags: Optional[List[str]] = None) -> str:
    """Bring libgdn.so and the binding's extension up to date, side by side. The library does not need the
    extension (Python's and PyTorch's headers): where that fails, the error comes after the library is in place."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        ext = ex.submit(_compile_ext, verbose) if force or ext_is_stale() else None
        build_lib(force, verbose, extra_flags)
        if ext is not None:
            _link_ext(ext.result(), verbose)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
