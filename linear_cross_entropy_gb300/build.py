"""Build libcce.so (the C-ABI library) in-tree with nvcc for sm_103a.

    python linear_cross_entropy_gb300/build.py [--verbose-ptxas]

(run by path: importing the package loads the library this script builds)

Each translation unit is compiled in parallel, then linked into
linear_cross_entropy_gb300/libcce.so against the shared CUDA runtime (the
one PyTorch loads), so both use the same runtime state.  csrc/binding.cpp
becomes the Python module _native.so beside it (g++, against this Python's and
PyTorch's headers), which calls libcce.so.  It works with that Python and that
PyTorch only, so their versions are kept beside the objects.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libcce.so")
NATIVE = os.path.join(PKG, "_native.so")
BUILT_FOR = os.path.join(BUILD, "native_for.txt")
COMMAND = "python linear_cross_entropy_gb300/build.py"
SOURCES = ("cce_api.cu", "gemm_kernels.cu", "cce_noalloc.cu", "cce_sort.cu", "cce_flce.cu", "grad_clip.cu",
           "norm_api.cu") + tuple(f"norm_{p}_{t}.cu" for p in ("fwd", "bwd")
                                  for t in ("bf16", "f16", "f32", "f32_bf16", "f32_f16"))
BINDING = "binding.cpp"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags(verbose_ptxas: bool):
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def _deps_mtime() -> float:
    paths = [os.path.join(d, p) for d in (CSRC, INCLUDE) for p in os.listdir(d)] + [__file__]
    return max(os.path.getmtime(p) for p in paths if os.path.isfile(p))


def versions() -> str:
    """What _native.so is bound to."""
    import torch
    return f"{sys.implementation.cache_tag}, torch {torch.__version__}"


def built_for() -> str:
    """versions() when _native.so was linked, "" if that is not known."""
    try:
        with open(BUILT_FOR) as f:
            return f.read()
    except FileNotFoundError:
        return ""


def up_to_date() -> bool:
    return built_for() == versions() and all(os.path.exists(p) and os.path.getmtime(p) >= _deps_mtime() for p in (LIB, NATIVE))


def _torch_flags():
    """Compile and link flags of a Python module over PyTorch."""
    import torch
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [sysconfig.get_paths()["include"], os.path.join(base, "include"),
               os.path.join(base, "include", "torch", "csrc", "api", "include"), os.path.join(cuda, "include")]
    compile_flags = ["-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
                     f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for d in include:
        compile_flags += ["-isystem", d]
    link_flags = ["-L" + os.path.join(base, "lib"), "-ltorch", "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda"]
    return compile_flags, link_flags


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = _flags(verbose_ptxas)

    torch_compile, torch_link = _torch_flags()
    cxx = os.environ.get("CXX") or "g++"

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc] + flags if src.endswith(".cu") else [cxx] + torch_compile
        r = subprocess.run(cmd + ["-c", os.path.join(CSRC, src), "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose_ptxas:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    def link(cmd, out):
        tmp = out + ".tmp"
        r = subprocess.run(cmd + ["-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, out)

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        *objs, binding = ex.map(compile_one, SOURCES + (BINDING,))
    link([cc] + ARCH + ["-shared", "--cudart", "shared"] + objs, LIB)
    link([cxx, "-shared", binding, "-L" + PKG, "-l:libcce.so", "-Wl,-rpath,$ORIGIN"] + torch_link, NATIVE)
    with open(BUILT_FOR, "w") as f:
        f.write(versions())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose_ptxas="--verbose-ptxas" in sys.argv))
