"""Build the sm_100a shared library librawint4_moe.so in-tree.

Usage: python -m int4_quantised_moe_b200.build  (or call build()).
The library is a plain C ABI (include/rawint4_moe.h); nvcc cross-compiles it
without a GPU. Beside it goes a small CPython extension, the quick way into the
operators around the layer. It is compiled against the installed Python and
torch, whose versions stand in its file name: another version finds no
extension of its own, never a wrong one, and every call then goes through
ctypes.
"""

from __future__ import annotations

import os
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "librawint4_moe.so")
FASTCALL_SOURCE = os.path.join(CSRC, "fastcall.cpp")
SOURCES = ["api.cu", "gemm_pair.cu", "gemm_tm.cu", "gemm_pair_narrow.cu", "gemm_tm_narrow.cu", "skinny.cu", "route.cu",
           "aux.cu", "prof.cu", "noalloc.cu", "router.cu", "select.cu", "select_f32.cu", "select_bf16.cu",
           "select_f16.cu", "norm.cu", "norm_fwd.cu", "norm_bwd_f32.cu", "norm_bwd_bf16.cu", "norm_bwd_f16.cu", "ckpt8.cu"]
HEADERS = ["common.cuh", "gemm.cuh", "skinny.cuh", "route.cuh", "aux.cuh", "prof.cuh", "router.cuh", "rows.cuh", "select.cuh",
           "select_kernels.cuh", "norm.cuh", "norm_kernels.cuh"]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _older(built: str, sources) -> bool:
    """Whether `built` is missing or older than one of its sources."""
    if not os.path.exists(built):
        return True
    t = os.path.getmtime(built)
    return any(os.path.getmtime(d) > t for d in sources if os.path.exists(d))


def _header() -> str:
    return os.path.join(ROOT, "include", "rawint4_moe.h")


def _library_stale() -> bool:
    return _older(LIB, [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [_header()])


def _fastcall_stale() -> bool:
    return _older(fastcall_path(), [FASTCALL_SOURCE, _header()])


def fastcall_path() -> str:
    """Where the extension for this Python and torch lies."""
    import sysconfig

    import torch
    return os.path.join(HERE, f"_fastcall-torch{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def _build_fastcall(verbose: bool) -> None:
    """Compile fastcall.cpp against this Python and torch, linked to LIB beside it."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    path = fastcall_path()
    tmp = path + ".tmp"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *[f"-isystem{p}" for p in include], FASTCALL_SOURCE, "-o", tmp, f"-L{HERE}", "-l:librawint4_moe.so",
           "-Wl,-rpath,$ORIGIN", f"-L{os.path.join(root, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch", "-ltorch_cpu",
           "-ltorch_cuda", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, path)


def _build_library(verbose: bool) -> None:
    objdir = os.path.join(HERE, "_build")
    os.makedirs(objdir, exist_ok=True)
    from concurrent.futures import ThreadPoolExecutor

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        cmd = [_nvcc(), *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
        return obj

    # independent translation units compile in parallel
    with ThreadPoolExecutor(max_workers=max(1, min(len(SOURCES), os.cpu_count() or 1))) as pool:
        objs = list(pool.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [_nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs]
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is missing or older than its sources (force: everything). Without a host compiler or
    torch's headers the library stands alone, with a warning."""
    if force or _library_stale():
        _build_library(verbose)
    try:
        if force or _fastcall_stale():
            _build_fastcall(verbose)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        warnings.warn(f"the quick way into the operators around the layer was not built ({e}); their calls go "
                      "through ctypes", RuntimeWarning)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
