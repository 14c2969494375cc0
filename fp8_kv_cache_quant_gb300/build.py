"""Build libfp8kv.so in-tree with nvcc for sm_103a (no cmake, one -gencode), and the binding's
compiled part, _binding.so, with the host compiler against torch's headers.

Each CUDA translation unit is compiled in parallel, then linked into
``fp8_kv_cache_quant_gb300/libfp8kv.so``.  The CUDA runtime is linked statically;
the driver API is reached through the runtime's entry-point query, so the library
loads on a machine without a GPU driver (the symbol checks of the CPU tests).
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
OUT = os.path.join(PKG, "libfp8kv.so")
BINDING = os.path.join(PKG, "_binding.so")
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include")]
SOURCES = ["abi.cu", "kv_quant_cache.cu", "decode_attn.cu", "decode_tc.cu", "prefill_attn.cu", "decode_noalloc.cu",
           "rope_cache.cu", "block_prefill.cu", "block_decode.cu"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _stale(srcs, out) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "fp8kv.h"), __file__]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _compile_binding(obj: str):
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    dirs = [sysconfig.get_paths()["include"], inc, os.path.join(inc, "torch", "csrc", "api", "include")]
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *("-isystem" + d for d in dirs),
           "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling binding.cpp failed:\n{r.stdout}\n{r.stderr}")


def _link_binding(obj: str):
    """Against libfp8kv.so beside it and torch's libraries (those that torch has loaded already)."""
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX") or "g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libfp8kv.so", "-L" + lib, "-lc10",
           "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking _binding.so failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = False, force: bool = False, extra_flags=()) -> str:
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    if not force and not _stale(srcs, OUT) and not _stale(srcs, BINDING):
        return OUT
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    binding_obj = os.path.join(BUILD_DIR, "binding.o")
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        binding = ex.submit(_compile_binding, binding_obj)
        objs = list(ex.map(compile_one, srcs))
        binding.result()
    tmp = OUT + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OUT)
    _link_binding(binding_obj)
    return OUT


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(verbose=v or bool(extra), force=True, extra_flags=extra))
