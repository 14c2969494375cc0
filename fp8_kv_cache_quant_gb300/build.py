"""Build libfp8kv.so in-tree with nvcc for sm_103a (no cmake, one -gencode), and the binding's
compiled part, binding_path(), with the host compiler against Python's and torch's headers.  The
library needs neither of them: it is in place before the binding is built, and by itself with --library.

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
BUILD_DIR = os.path.join(ROOT, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include")]
SOURCES = ["abi.cu", "kv_quant_cache.cu", "decode_attn.cu", "decode_tc.cu", "prefill_attn.cu", "decode_noalloc.cu",
           "rope_cache.cu", "block_prefill.cu", "block_decode.cu", "block_evict.cu", "block_weights.cu", "block_shared.cu"]


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _stale(out, sources) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    deps = [os.path.join(CSRC, f) for f in sources] + [os.path.join(ROOT, "include", "fp8kv.h"), __file__]
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def binding_path() -> str:
    """The compiled binding of this Python and this torch, whose C++ interfaces it is built against."""
    import sysconfig

    import torch
    return os.path.join(PKG, f"_binding-torch-{torch.__version__}-{sysconfig.get_config_var('SOABI')}.so")


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
    out = binding_path()
    tmp = out + ".tmp"
    cmd = [os.environ.get("CXX") or "g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libfp8kv.so", "-L" + lib, "-lc10",
           "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"linking the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def build(verbose: bool = False, force: bool = False, extra_flags=(), library_only: bool = False) -> str:
    srcs = [s for s in SOURCES if os.path.exists(os.path.join(CSRC, s))]
    library = force or _stale(OUT, [f for f in os.listdir(CSRC) if f != "binding.cpp"])
    binding = not library_only and (force or _stale(binding_path(), ["binding.cpp"]))
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc() if library else None

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
        compiled = ex.submit(_compile_binding, binding_obj) if binding else None
        if library:
            objs = list(ex.map(compile_one, srcs))
            tmp = OUT + ".tmp"
            cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp, OUT)
        if binding:
            try:
                compiled.result()
                _link_binding(binding_obj)
            except RuntimeError as e:
                raise RuntimeError(f"{OUT} is built, the compiled binding is not: {e}") from e
    return OUT


if __name__ == "__main__":
    v = "-v" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas" in sys.argv else []
    print(build(verbose=v or bool(extra), force=True, extra_flags=extra, library_only="--library" in sys.argv))
