"""Builds the CUDA library in-tree: ``_build/libbsa_topk_<machine>.so``.

The library is compiled for sm_103a only (GB300), from the sources in
``csrc/``, with nvcc.  Translation units compile in parallel; the link pulls
in the static CUDA runtime so the library loads without a CUDA runtime on the
loader path.  Beside it, ``_build/bsa_binding.so`` is the Python module that
checks and marshals the arguments of the cache operators (host compiler,
PyTorch's headers).  Run ``python -m block_sparse_attention_topk_gb300.build`` or
call ``build()``.
"""
from __future__ import annotations

import os
import platform
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB_NAME = f"libbsa_topk_{platform.machine()}.so"
LIB_PATH = os.path.join(BUILD, LIB_NAME)
SOURCES = ["bsa_select.cu", "bsa_table.cu", "bsa_capi.cu", "bsa_noalloc.cu", "bsa_attention.cu",
           "bsa_rope.cu", "bsa_append.cu", "bsa_attention_q8.cu"]
BINDING = "bsa_binding.cpp"
BINDING_PATH = os.path.join(BUILD, f"bsa_binding_{platform.machine()}.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + [BINDING]]
    files += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    files.append(os.path.join(INCLUDE, "bsa_topk.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(BINDING_PATH):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(BINDING_PATH))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-I", INCLUDE, *extra_flags]
    objs = []

    def compile_binding():
        import torch
        torch_dir = os.path.dirname(torch.__file__)
        obj = os.path.join(BUILD, f"bsa_binding_{platform.machine()}.o")
        cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-c",
               "-D_GLIBCXX_USE_CXX11_ABI=" + str(int(torch._C._GLIBCXX_USE_CXX11_ABI)),
               "-isystem", os.path.join(torch_dir, "include"),
               "-isystem", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, BINDING), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"the host compiler failed on {BINDING}:\n{res.stdout}\n{res.stderr}")
        return obj, os.path.join(torch_dir, "lib")

    def compile_one(src):
        obj = os.path.join(BUILD, f"{os.path.splitext(src)[0]}_{platform.machine()}.o")
        cmd = [cc, *common, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            print(res.stdout, res.stderr, flush=True)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as pool:
        binding = pool.submit(compile_binding)
        objs = list(pool.map(compile_one, SOURCES))
        binding_obj, torch_lib = binding.result()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB_PATH)
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "c++", "-shared", "-o", tmp, binding_obj, "-L", BUILD,
           f"-l:{LIB_NAME}", "-L", torch_lib, "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_lib}"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"linking {BINDING} failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []))
