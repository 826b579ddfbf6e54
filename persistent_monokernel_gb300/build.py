"""Build liblf.so (the CUDA library behind include/lf.h) in-tree with nvcc, and _lft.so (KV4Cache's calls, for Python).

    python -m persistent_monokernel_gb300.build

Compiles each .cu translation unit for sm_103a in parallel, then links a
shared library with the CUDA runtime linked statically.  No other library is
linked: the batched prefill's GEMMs are this library's own tcgen05 kernels,
and the tensor maps are encoded through the runtime's driver entry point.
_lft.so is host code against PyTorch's headers and does not link liblf.so.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "liblf.so")
EXT = os.path.join(HERE, "_lft.so")
SOURCES = ["lf_kernel.cu", "lf_api.cu", "lf_noalloc.cu", "lf_syncbench.cu", "lf_prefill.cu", "lf_gemm.cu", "lf_attn_tc.cu",
           "lf_kv4.cu", "lf_kv4_tc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps() -> list:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(ROOT, "include", "lf.h"))
    files.append(os.path.abspath(__file__))
    return files


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(EXT)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    def compile_ext():
        # torch's place is looked up, not imported
        torch = importlib.util.find_spec("torch").submodule_search_locations[0]
        tmp = EXT + f".tmp{os.getpid()}"
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
               "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(torch, "include"),
               "-I" + os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               "-I" + os.path.join(os.path.dirname(os.path.dirname(cc)), "include"),
               os.path.join(CSRC, "lf_torch.cpp"), "-o", tmp, "-L" + os.path.join(torch, "lib"),
               "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed for lf_torch.cpp:\n{r.stdout}\n{r.stderr}")
        return tmp

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        ext = ex.submit(compile_ext)
        objs = list(ex.map(compile_one, SOURCES))
        ext = ext.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(ext, EXT)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
