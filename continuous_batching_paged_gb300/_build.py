"""Build libcb.so in-tree with nvcc for sm_103a (no cmake, no torch extension machinery), and the
Python extension that binds its per-step calls to torch tensors.

Each .cu file compiles to an object in parallel; the objects link into one shared library
with the CUDA runtime linked statically, so loading the library needs no GPU or driver.  The
extension (csrc/cb_torch.cpp) compiles beside them with the host compiler against the headers of the
installed Python and torch, and links to libcb.so next to it.  The library builds and loads without
torch; the extension is built where there is one.
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


def _is_old(path: str, deps: list[str]) -> bool:
    """Whether `path` is missing or older than one of `deps` (or this file)."""
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in [*deps, os.path.abspath(__file__)])


def _in(folder: str, suffixes) -> list[str]:
    return [os.path.join(folder, f) for f in os.listdir(folder) if f.endswith(suffixes)]


def library_is_stale() -> bool:
    return _is_old(LIB, _in(CSRC, (".cu", ".cuh", ".h")) + _in(INCLUDE, ".h"))


def _ext_stamp() -> str:
    """What the extension is compiled for, beside its sources: this Python and the installed torch."""
    torch = _torch_dir()
    with open(os.path.join(torch, "version.py")) as f:
        return f"{sys.version}\n{torch}\n{f.read()}"


def _ext_stamp_path() -> str:
    return os.path.join(BUILD_DIR, "cb_torch.stamp")


def extension_is_stale() -> bool:
    """Whether the extension is missing, older than its sources, or compiled for another Python or
    torch than those that are here."""
    if _is_old(EXT, [EXT_SOURCE, *_in(INCLUDE, ".h")]):
        return True
    if _torch_dir() is None:
        return False
    try:
        with open(_ext_stamp_path()) as f:
            return f.read() != _ext_stamp()
    except FileNotFoundError:  # (built files that came without the build's folder)
        return False


def is_stale() -> bool:
    """Whether build() has something to do (without torch there is no extension to build)."""
    return library_is_stale() or (_torch_dir() is not None and extension_is_stale())


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


def _torch_dir() -> str | None:
    """Where torch is installed (None: it is not)."""
    spec = importlib.util.find_spec("torch")
    return None if spec is None else list(spec.submodule_search_locations)[0]


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
    with open(_ext_stamp_path(), "w") as f:
        f.write(_ext_stamp())


def build_library(verbose: bool = False) -> str:
    """Compile every kernel source and link libcb.so; returns its path.  Needs no torch."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        results = list(ex.map(_compile, srcs))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [_nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *[o for o, _ in results],
           "-ldl", "-lpthread", "-lrt"]
    _run(cmd, "link")
    os.replace(tmp, LIB)
    return LIB


def build_extension() -> str:
    """Compile and link the extension against libcb.so, which must be there; returns its path."""
    if _torch_dir() is None:
        raise RuntimeError("torch not found: the Python binding needs its headers")
    os.makedirs(BUILD_DIR, exist_ok=True)
    _link_ext(_compile_ext())
    return EXT


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is missing or older than its sources (force: everything): libcb.so and, where
    torch is installed, the extension.  Returns the library's path.  The library is linked whatever
    becomes of the extension: the allocator, the scheduler and the C ABI need neither torch nor its
    headers."""
    lib = force or library_is_stale()
    ext = _torch_dir() is not None and (force or extension_is_stale())
    if ext:
        os.makedirs(BUILD_DIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=1) as ex:
        obj = ex.submit(_compile_ext) if ext else None  # (beside the kernels)
        if lib:
            build_library(verbose)
        if obj is not None:
            _link_ext(obj.result())
    return LIB
