"""Build the C-ABI shared library libbf16_linear.so in-tree with nvcc (sm_103a only).

    python -m moe_router_gemm_gb300.build [--force]

Beside it, a small module that marshals calls from PyTorch tensors in C++
(csrc/torch_calls.cpp), where the installed PyTorch's headers allow.

Each translation unit compiles in parallel to _build/*.o, then one link step
produces moe_router_gemm_gb300/libbf16_linear.so (CUDA runtime linked
statically, so the library needs only the driver at run time).
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import hashlib
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libbf16_linear.so")

SOURCES = ["api.cu", "plan.cpp", "dotprod.cu", "dotprod_f32.cu", "splitk.cu", "tile.cu", "tile_t.cu", "stream.cu", "noalloc.cu", "tile2.cu", "warprow.cu", "warpmma.cu", "warpmma_ks.cu", "dotmma.cu", "fp8.cu", "mxfp8.cu", "probe.cu", "mxfp4.cu", "mxfp4_pair.cu", "mxfp4_split.cu",
           "norm.cu", "route.cu", "api_moe.cu"]
HEADERS = ["common.cuh", "kernels.h", "moe.h", "dotprod.cuh", "tile.cuh", "mxfp4.cuh", "dispatch_table.inc"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC = os.environ.get("NVCC", "nvcc")
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-I" + INCLUDE, "-I" + CSRC]


def _inputs():
    return ([os.path.join(CSRC, s) for s in SOURCES] + [os.path.join(CSRC, h) for h in HEADERS]
            + [os.path.join(INCLUDE, "bf16_linear.h"), os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _compile(src: str, extra: list[str]) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    if src.endswith(".cpp"):
        cmd = [NVCC, *FLAGS, *extra, "-x", "c++", "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


CALLS_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared"]


def _calls_stem() -> str:
    import sysconfig

    import torch
    return "_torch_calls_" + "".join(c if c.isalnum() else "_" for c in f"{torch.__version__}_{sysconfig.get_config_var('SOABI')}") + "_"


def calls_path() -> str:
    """The compiled marshalling module (csrc/torch_calls.cpp).  It uses PyTorch's and Python's C++ types and the library's
    argument lists, so its name says which release, which Python and which sources it was built from: a file that stands
    there is never one of another."""
    h = hashlib.sha256(" ".join(CALLS_FLAGS).encode())
    for path in (os.path.join(CSRC, "torch_calls.cpp"), os.path.join(INCLUDE, "bf16_linear.h")):
        with open(path, "rb") as f:
            h.update(f.read())
    return os.path.join(PKG, f"{_calls_stem()}{h.hexdigest()[:16]}.so")


def build_calls(force: bool = False) -> str | None:
    """Compile the marshalling module for the installed PyTorch; None where it cannot be (the binding then calls the library
    through ctypes alone)."""
    try:
        import sysconfig

        import torch
        out = calls_path()
        if not force and os.path.exists(out):
            return out
        root = os.path.dirname(torch.__file__)
        cuda = os.environ.get("CUDA_HOME") or "/usr/local/cuda"
        inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
        libs = os.path.join(root, "lib")
        tmp = out + f".tmp{os.getpid()}"
        cmd = ["g++", *CALLS_FLAGS, f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               *("-I" + i for i in inc), os.path.join(CSRC, "torch_calls.cpp"), "-o", tmp, "-L" + libs, "-Wl,-rpath," + libs,
               "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            print(f"torch_calls.cpp does not build, calls go through ctypes:\n{r.stderr[-2000:]}", file=sys.stderr)
            return None
        os.replace(tmp, out)
        for name in os.listdir(PKG):  # of earlier sources
            if name.startswith(_calls_stem()) and name.endswith(".so") and name != os.path.basename(out):
                with contextlib.suppress(FileNotFoundError):  # (another build took it)
                    os.remove(os.path.join(PKG, name))
        return out
    except (ImportError, OSError) as e:
        print(f"torch_calls.cpp is not built, calls go through ctypes: {e}", file=sys.stderr)
        return None


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        build_calls()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(build_calls, force)
        objs = list(ex.map(lambda s: _compile(os.path.join(CSRC, s), extra), SOURCES))
        calls.result()  # (raises what build_calls did not handle)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    print(build(force=force, verbose_ptxas="--ptxas" in sys.argv))
