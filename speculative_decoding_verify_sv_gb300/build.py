"""Build libsv.so (the verify-step C ABI) in-tree with nvcc for sm_103a, and sv_binding.so (the
compiled Python calls of the operators around the KV cache) with g++ against the installed torch.

Each translation unit compiles in parallel to an object file; one nvcc call links the
shared library.  Objects are rebuilt only when a source or header is newer.
``python -m speculative_decoding_verify_sv_gb300.build`` runs it from the shell.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
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
LIB = os.path.join(BUILD, "libsv.so")
BINDING = os.path.join(BUILD, "sv_binding.so")

SOURCES = ["sv_api.cu", "attention.cu", "attention_tc.cu", "attention_tc_window.cu", "attention_tc_window_paged.cu", "window_attention.cu", "window_attention_f32.cu", "stacked_attention.cu", "stacked_units.cu", "joined_units.cu",
           "own_units.cu", "listed_units.cu", "warp_units.cu", "own_warps.cu", "pages.cu", "page_scores_tc.cu",
           "accept.cu", "accept_recursive.cu", "commit.cu", "ngram.cu", "lm_head.cu", "tables.cu", "qk_norm_rope.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                 "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _newest_dep() -> float:
    deps = glob.glob(os.path.join(CSRC, "*")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(d) for d in deps)


def _compile(nvcc: str, src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    log = obj + ".ptxas.txt"
    if os.path.exists(obj) and os.path.getmtime(obj) >= _newest_dep():
        return obj
    cmd = [nvcc, *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(log, "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr[-6000:]}")
    os.replace(obj + ".tmp", obj)
    return obj


def _binding_flags():
    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    cflags = ["-O2", "-std=c++17", "-fPIC", "-Wno-psabi",
              f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
              "-isystem", os.path.join(base, "include"),
              "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
              "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"]]
    libs = ["-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
            "-L", BUILD, "-l:libsv.so", "-Wl,-rpath,$ORIGIN"]
    return cflags, libs


def _compile_binding() -> str:
    """sv_binding.o: independent of libsv.so, so that it compiles beside the kernels."""
    src, obj = os.path.join(CSRC, "binding.cpp"), os.path.join(BUILD, "binding.o")
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "sv.h")))
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj
    cflags, _ = _binding_flags()
    cmd = ["g++", *cflags, "-c", src, "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stderr[-6000:]}")
    os.replace(obj + ".tmp", obj)
    return obj


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every translation unit for sm_103a and link libsv.so; returns its path."""
    os.makedirs(BUILD, exist_ok=True)
    if force:
        for f in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(f)
    nvcc = _nvcc()
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        objs = list(ex.map(lambda s: _compile(nvcc, s), SOURCES))
        binding = binding.result()
    if not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
        os.replace(tmp, LIB)
    if not os.path.exists(BINDING) or os.path.getmtime(BINDING) < max(os.path.getmtime(binding), os.path.getmtime(LIB)):
        _, libs = _binding_flags()
        tmp = BINDING + f".{os.getpid()}.tmp"
        r = subprocess.run(["g++", "-shared", "-o", tmp, binding, *libs], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
        os.replace(tmp, BINDING)
    if verbose:
        for s in SOURCES:
            p = os.path.join(BUILD, os.path.splitext(s)[0] + ".o.ptxas.txt")
            if os.path.exists(p):
                print(open(p).read())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
