"""Build libmm3idx.so in-tree with nvcc for sm_103a, and the Python binding of
the operators that use the selection (_binding.so) with the host compiler.

Each translation unit compiles in parallel; the shared library links the CUDA
runtime statically and resolves the driver's tensor-map encoder at run time,
so loading it needs no GPU and no libcuda.

    python sparse_attention_block_paged_gb300/build.py [-v]
"""

from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "_lib")
LIB = os.path.join(OUT_DIR, "libmm3idx.so")
SOURCES = ["api.cu", "decode.cu", "decode_fp4.cu", "prefill.cu", "select.cu", "dequant.cu",
           "sparse_table.cu", "api_serving.cu", "attention.cu", "attention_bf16.cu",
           "attention_fp16.cu", "attention_bf16_e4m3.cu", "attention_fp16_e4m3.cu",
           "attention_bf16_e4m3_scaled.cu", "attention_fp16_e4m3_scaled.cu", "evict.cu",
           "verify.cu", "api_pages.cu", "append.cu", "pages.cu"]
HEADERS = ["internal.h", "ptx.cuh", "warp_select.cuh", "decode_common.cuh", "nvfp4.cuh",
           "serving.h", "attention.cuh", "pages.h"]

BINDING = os.path.join(OUT_DIR, "_binding.so")

CXX = os.environ.get("CXX", "g++")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, verbose):
    obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
    deps = [os.path.join(CSRC, src)] + [os.path.join(CSRC, h) for h in HEADERS] + [
        os.path.join(ROOT, "include", "mm3idx.h")]
    if not _stale(obj, deps):
        return obj, ""
    cmd = [NVCC, *ARCH, *FLAGS, "-Xptxas", "-v", "-c", os.path.join(CSRC, src), "-o", obj + ".tmp"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj, r.stderr if verbose else ""


def _compile_binding():
    """binding.cpp against torch's headers (torch itself is not imported)."""
    src, obj = os.path.join(CSRC, "binding.cpp"), os.path.join(OUT_DIR, "binding.o")
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    if _stale(obj, [src, os.path.join(ROOT, "include", "mm3idx.h"),
                    os.path.join(torch, "version.py")]):
        cuda = os.path.dirname(os.path.dirname(NVCC))
        cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-c", src, "-o", obj + ".tmp",
               "-I", sysconfig.get_paths()["include"], "-I", os.path.join(torch, "include"),
               "-I", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               "-I", os.path.join(cuda, "include")]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{CXX} failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
        os.replace(obj + ".tmp", obj)
    return obj, os.path.join(torch, "lib")


def _link_binding(obj, torch_lib):
    if not _stale(BINDING, [obj, LIB]):
        return
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [CXX, "-shared", obj, "-o", tmp, "-L", OUT_DIR, "-l:libmm3idx.so", "-L", torch_lib,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(lambda s: _compile(s, verbose), SOURCES))
        binding_obj, torch_lib = binding.result()
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            if log:
                print(log)
    if _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", *objs, "-o", tmp,
               "-Xlinker", "-soname=libmm3idx.so"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _link_binding(binding_obj, torch_lib)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
