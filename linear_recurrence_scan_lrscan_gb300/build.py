"""Build liblrscan.so in-tree with nvcc for sm_103a (GB300).

Each translation unit is compiled in parallel, then linked into one shared
library under ``_build/``.  No CMake; only nvcc and the host compiler.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "liblrscan.so")
BINDING = os.path.join(BUILD, "lrscan_layer.so")  # Python binding of the operators around the scan
SOURCES = ["lrscan_abi.cu", "kernels_window.cu", "kernels_window_state.cu", "kernels_chunk.cu", "kernels_complex.cu", "kernels_complex_state.cu", "kernels_complex_chunk.cu", "kernels_stream.cu", "kernels_gated.cu", "kernels_gates.cu", "kernels_conv.cu", "kernels_embed.cu", "layer_abi.cu", "noalloc_chunk.cu", "host_pipeline.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build liblrscan.so")


def cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def compile_flags(extra=()) -> list[str]:
    return [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
            "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}", *extra]


def binding_command(out: str) -> list[str]:
    """The host compiler's command for layer_binding.cpp, against this Python and this torch."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    cuda = os.path.dirname(cuda_lib_dir(_nvcc()))
    includes = [sysconfig.get_paths()["include"], *cpp_extension.include_paths(), os.path.join(cuda, "include"), INCLUDE]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *[x for i in includes for x in ("-isystem", i)], os.path.join(CSRC, "layer_binding.cpp"), "-o", out,
            f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    headers.append(os.path.join(INCLUDE, "lrscan.h"))
    objs, jobs = [], []
    for src in SOURCES:
        path = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [path, *headers]):
            jobs.append([nvcc, *compile_flags(extra_flags), "-c", path, "-o", obj])

    binding = BINDING + f".tmp{os.getpid()}"
    bind = force or _stale(BINDING, [os.path.join(CSRC, "layer_binding.cpp"), os.path.join(INCLUDE, "lrscan.h")])
    if bind:
        jobs.append(binding_command(binding))

    def run(cmd):
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"compiling failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr, file=sys.stderr)
        return r

    with cf.ThreadPoolExecutor(max_workers=max(1, len(jobs))) as ex:
        list(ex.map(run, jobs))
    if bind:
        os.replace(binding, BINDING)
    if force or jobs or _stale(LIB, objs):
        libdir = cuda_lib_dir(nvcc)
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "shared",
             f"-L{libdir}", "-Xlinker", f"-rpath,{libdir}"])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
