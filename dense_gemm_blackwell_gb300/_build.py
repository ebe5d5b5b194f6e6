"""Build the CUDA library in-tree: nvcc, sm_103a only, sources compiled in parallel.

Produces ``dense_gemm_blackwell_gb300/libdgb_gemm.so`` (git-ignored).  The
library links the CUDA runtime statically and resolves the driver's tensor-map
encoder at run time, so it loads on machines without a GPU.  Next to it,
``_tensor_facts.so``: a small Python extension for the serving operators'
binding (the CUDA library itself knows neither Python nor torch).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libdgb_gemm.so")
FACTS = os.path.join(PKG, "_tensor_facts.so")
BUILD_DIR = os.path.join(PKG, "_build")

SOURCES = ["kernels_single.cu", "kernels_persistent.cu", "kernels_fp8.cu", "kernels_mx.cu", "gemm_api.cu",
           "schedule_model.cu", "lora.cu", "lora_skinny.cu", "qk_norm_rope.cu", "paged_attn_api.cu", "paged_attn_bf16.cu", "paged_attn_f16.cu",
           "paged_attn_bf16_e4m3.cu", "paged_attn_f16_e4m3.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the CUDA toolkit is required to build the library")


def torch_headers():
    """Folder of the installed torch if it and Python come with C++ headers, else None."""
    try:
        import torch
    except ImportError:
        return None
    root = os.path.dirname(os.path.abspath(torch.__file__))
    needed = (os.path.join(root, "include", "torch", "csrc", "autograd", "python_variable.h"),
              os.path.join(sysconfig.get_paths()["include"], "Python.h"))
    return root if all(os.path.exists(f) for f in needed) and shutil.which("g++") else None


def build_facts() -> None:
    """Compile the tensor_facts extension against the installed torch; without its headers the binding asks in Python."""
    root = torch_headers()
    if root is None:
        return
    tmp = FACTS + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(root, "include"),
           "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"), os.path.join(CSRC, "tensor_facts.cpp"), "-o", tmp,
           "-L" + os.path.join(root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath," + os.path.join(root, "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("g++ failed for tensor_facts.cpp:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, FACTS)


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    files += [os.path.join(INCLUDE, f) for f in ("gemm.h", "serving.h")]
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    outputs = [LIB] + ([FACTS] if torch_headers() else [])
    if not all(os.path.exists(f) for f in outputs):
        return False
    t = min(os.path.getmtime(f) for f in outputs)
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, ptxas_verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        facts = ex.submit(build_facts)
        results = list(ex.map(compile_one, SOURCES))
        facts.result()
    if verbose or ptxas_verbose:
        for _, log in results:
            if log:
                sys.stderr.write(log)
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_verbose="-v" in sys.argv))
