"""Build libcb.so in-tree with nvcc for sm_103a (no cmake, no torch extension machinery), and the
Python extension that binds its per-step calls to torch tensors.

Each .cu file compiles to an object in parallel; the objects link into one shared library
with the CUDA runtime linked statically, so loading the library needs no GPU or driver.  The
extension (csrc/cb_torch.cpp) compiles beside them with the host compiler against the headers of the
installed Python and torch, and links to libcb.so next to it.
"""
from __future__ import annotations

import concurrent.futures
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(os.path.dirname(PKG), "include")
LIB = os.path.join(PKG, "libcb.so")
EXT = os.path.join(PKG, "_cb_torch.so")
EXT_SOURCE = os.path.join(CSRC, "cb_torch.cpp")
BUILD_DIR = os.path.join(PKG, "_build")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: libcb needs the CUDA toolkit to build")


def sources() -> list[str]:
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps() -> list[str]:
    out = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    out += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    out.append(os.path.abspath(__file__))
    return out


def is_stale() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(EXT)):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found: the Python binding needs its headers")
    return list(spec.submodule_search_locations)[0]


def _compile_ext() -> str:
    obj = os.path.join(BUILD_DIR, "cb_torch.o")
    torch = _torch_dir()
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    inc = [os.path.join(torch, "include"),
           os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], cuda]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC",
          *[x for i in inc for x in ("-isystem", i)], "-c", EXT_SOURCE, "-o", obj],
         "compiling cb_torch.cpp")
    return obj


def _link_ext(obj: str) -> None:
    lib = os.path.join(_torch_dir(), "lib")
    tmp = EXT + f".tmp{os.getpid()}"
    _run([os.environ.get("CXX", "g++"), "-shared", obj, "-o", tmp, "-L", PKG, "-l:libcb.so",
          "-Wl,-rpath,$ORIGIN", "-L", lib, "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
          "-lc10_cuda", "-lc10"], "linking _cb_torch.so")
    os.replace(tmp, EXT)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile every kernel source and link libcb.so; returns its path."""
    if not force and not is_stale():
        return LIB
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        ext = ex.submit(_compile_ext)
        results = list(ex.map(_compile, srcs))
        ext_obj = ext.result()
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *[o for o, _ in results],
           "-ldl", "-lpthread", "-lrt"]
    _run(cmd, "link")
    os.replace(tmp, LIB)
    _link_ext(ext_obj)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
