"""Build liblf.so (the CUDA library behind include/lf.h) in-tree with nvcc, and _lft.so (KV4Cache's calls, for Python).

    python -m persistent_monokernel_gb300.build

Compiles each .cu translation unit for sm_103a in parallel, then links a
shared library with the CUDA runtime linked statically.  No other library is
linked: the batched prefill's GEMMs are this library's own tcgen05 kernels,
and the tensor maps are encoded through the runtime's driver entry point.
_lft.so is host code against PyTorch's headers and does not link liblf.so, nor
liblf.so it: without PyTorch the library is built all the same.
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
EXT, EXT_SOURCE = os.path.join(HERE, "_lft.so"), "lf_torch.cpp"
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


def _newer(target, sources) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in sources)


def lib_up_to_date() -> bool:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != EXT_SOURCE]
    return _newer(LIB, files + [os.path.join(ROOT, "include", "lf.h"), os.path.abspath(__file__)])


def _torch_place():
    """torch's folder, looked up and not imported; None where there is no torch."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec else None


def _ext_stamp(torch: str) -> str:
    """What _lft.so fits besides its sources: this Python, and this torch in this place."""
    with open(os.path.join(torch, "version.py")) as f:
        return f"{sys.version}\n{torch}\n{f.read()}"


def ext_up_to_date() -> bool:
    """True where there is no torch, too: nobody could use the module."""
    torch = _torch_place()
    if torch is None:
        return True
    if not _newer(EXT, [os.path.join(CSRC, EXT_SOURCE), os.path.join(ROOT, "include", "lf.h"), os.path.abspath(__file__)]):
        return False
    stamp = os.path.join(BUILD, "_lft.stamp")
    if not os.path.exists(stamp):
        return False
    with open(stamp) as f:
        return f.read() == _ext_stamp(torch)


def up_to_date() -> bool:
    return lib_up_to_date() and ext_up_to_date()


def _run(cmd, what, verbose=False):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed {what}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)


def _build_ext(cc) -> None:
    torch = _torch_place()
    tmp = EXT + f".tmp{os.getpid()}"
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
          "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(torch, "include"),
          "-I" + os.path.join(torch, "include", "torch", "csrc", "api", "include"),
          "-I" + os.path.join(os.path.dirname(os.path.dirname(cc)), "include"),
          os.path.join(CSRC, EXT_SOURCE), "-o", tmp, "-L" + os.path.join(torch, "lib"),
          "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"], f"for {EXT_SOURCE}")
    os.replace(tmp, EXT)
    with open(os.path.join(BUILD, "_lft.stamp"), "w") as f:
        f.write(_ext_stamp(torch))


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is not up to date.  liblf.so needs nvcc only; _lft.so is left out where there is no torch, and where
    it cannot be built that is raised once liblf.so stands."""
    lib, ext = force or not lib_up_to_date(), (force and _torch_place() is not None) or not ext_up_to_date()
    if not (lib or ext):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        _run([cc, *(["-Xptxas=-v"] if verbose else []), *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj],
             f"for {src}", verbose)
        return obj

    with ThreadPoolExecutor(len(SOURCES) + 1) as ex:
        module = ex.submit(_build_ext, cc) if ext else None
        if lib:
            objs = list(ex.map(compile_one, SOURCES))
            tmp = LIB + f".tmp{os.getpid()}"
            _run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], "to link liblf.so")
            os.replace(tmp, LIB)
        if module:
            module.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
