"""In-tree build of libkda.so for sm_103a (nvcc + g++, translation units compiled in parallel).

Loaded by file path from __graft_entry__.build(), so it imports nothing from the package.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libkda.so")
OPS = os.path.join(PKG, "_ops.so")     # the marshalling module of binding.py (csrc/torch_ops.cpp)
ROOT = os.path.dirname(PKG)

CUDA_SOURCES = ["api.cu", "chunk_prep.cu", "chunk_state.cu", "compose.cu", "boundary.cu", "noalloc.cu", "backward.cu", "reverse.cu",
                "gated_scan.cu", "gated_scan_backward.cu", "decode.cu", "block_norm.cu",
                "block_norm_forward_bf16.cu", "block_norm_forward_f16.cu", "block_norm_backward_bf16.cu",
                "block_norm_backward_f16.cu"]
CXX_SOURCES = ["plan.cpp"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libkda")


def _newest_input() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "kda.h"),
                                                                   os.path.abspath(__file__)]
    return max(os.path.getmtime(p) for p in paths if os.path.exists(p))


def _torch_dir():
    """torch's folder, found without importing it; None where there is no torch with CUDA (the C library needs none)."""
    spec = importlib.util.find_spec("torch")
    for path in (spec.submodule_search_locations or ()) if spec else ():
        if os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")):
            return path
    return None


def build(force: bool = False, verbose: bool = False, extra_nvcc=()) -> str:
    """Compile csrc/ into context_kda_gb300/libkda.so and, where torch is found, _ops.so, unless they are up to date."""
    torch = _torch_dir()
    made = (LIB, OPS) if torch else (LIB,)
    if not force and all(os.path.exists(p) and os.path.getmtime(p) >= _newest_input() for p in made):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    inc = ["-I", os.path.join(ROOT, "include")]
    jobs = []
    for src in CUDA_SOURCES:
        obj = os.path.join(BUILD, src + ".o")
        jobs.append([nvcc, *ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
                     "--expt-relaxed-constexpr", *inc, *extra_nvcc, "-c", os.path.join(CSRC, src), "-o", obj])
    for src in CXX_SOURCES:
        obj = os.path.join(BUILD, src + ".o")
        jobs.append(["g++", "-O2", "-std=c++17", "-fPIC", *inc, "-c", os.path.join(CSRC, src), "-o", obj])

    # torch's libraries are already loaded when the marshalling module is
    ops_obj = os.path.join(BUILD, "torch_ops.cpp.o")
    if torch:
        cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
        jobs.append(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-I", os.path.join(torch, "include"), "-I",
                     os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"), "-I",
                     sysconfig.get_paths()["include"], "-c", os.path.join(CSRC, "torch_ops.cpp"), "-o", ops_obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"build step failed: {' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return r

    with cf.ThreadPoolExecutor(max_workers=len(jobs)) as ex:
        list(ex.map(run, jobs))
    objs = [os.path.join(BUILD, s + ".o") for s in CUDA_SOURCES + CXX_SOURCES]
    tmp = LIB + f".tmp{os.getpid()}"
    run([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    if torch:
        tmp = OPS + f".tmp{os.getpid()}"
        run(["g++", "-shared", "-o", tmp, ops_obj, "-L", PKG, "-l:libkda.so", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(torch, "lib"),
             "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"])
        os.replace(tmp, OPS)
    return LIB
