"""Build libprune24.so in-tree for sm_103a (GB300) with nvcc.

Each .cu under csrc/ is compiled in parallel to an object file under _build/,
then all are linked into semi_structured_sparse_prune24_gb300/_lib/libprune24.so.
csrc/p24_torch.cpp, the binding's marshalling of torch tensors, is compiled beside them
(with torch's headers) and linked into _lib/_p24_torch.so, which uses libprune24.so; where that
fails libprune24.so is there all the same, and the build says so.
Nothing is installed outside the repository. Run: python semi_structured_sparse_prune24_gb300/build.py
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
BUILD = os.path.join(ROOT, "_build")
LIBDIR = os.path.join(PKG, "_lib")
LIB = os.path.join(LIBDIR, "libprune24.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; libprune24 needs the CUDA 13 toolkit")


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _compile(nvcc: str, src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    _run(cmd, f"nvcc failed on {src}")
    return obj


MARSHAL = os.path.join(LIBDIR, "_p24_torch.so")


def _compile_marshal(nvcc: str) -> str:
    import torch  # while the kernels are compiled: which ABI it has, and where it is

    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    obj = os.path.join(BUILD, "p24_torch.o")
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", f"-DP24_TORCH_VERSION=\"{torch.__version__}\"",
          f"-I{INCLUDE}", f"-I{inc}",
          f"-I{os.path.join(inc, 'torch', 'csrc', 'api', 'include')}", f"-I{cuda}", f"-I{sysconfig.get_paths()['include']}",
          "-c", os.path.join(CSRC, "p24_torch.cpp"), "-o", obj], "the host compiler failed on p24_torch.cpp")
    return obj


def _link_marshal(obj: str) -> None:
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = MARSHAL + ".tmp"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{LIBDIR}", "-lprune24", f"-L{lib}", "-ltorch_python",
          "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"], "link of p24_torch failed")
    os.replace(tmp, MARSHAL)


def build(verbose: bool = False) -> str:
    """Compile every CUDA source for sm_103a and link the shared library, then the binding's marshalling. Returns the
    library's path. Raises where either fails; the library does not need the marshalling."""
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        marshal = ex.submit(_compile_marshal, nvcc)
        objs = list(ex.map(lambda s: _compile(nvcc, s), srcs))
    libdir = _cuda_lib_dir(nvcc)
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           f"-L{libdir}", "-Xlinker", f"-rpath={libdir}", "-Xlinker", "-soname=libprune24.so"]
    _run(cmd, "link failed")
    os.replace(tmp, LIB)
    if os.path.exists(MARSHAL):
        os.remove(MARSHAL)  # of another build: not to be used if this one fails
    _link_marshal(marshal.result())
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
