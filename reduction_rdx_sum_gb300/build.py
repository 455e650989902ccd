"""Build librdx.so (the CUDA library) in-tree for sm_103a, and _marshal.so beside it.

Each translation unit is compiled by its own nvcc process (in parallel), then
linked into ``reduction_rdx_sum_gb300/librdx.so`` against the shared CUDA
runtime (the one PyTorch has already loaded, when it has).  ptxas resource
usage (registers, spills, shared memory) is written to ``_build/ptxas.txt``.
Nothing is rebuilt while the library is newer than every source and header.
``_marshal.so`` (csrc/marshal.cpp, g++ against PyTorch's headers) marshals the
arguments of the calls over heads from Python; it is compiled alongside where
PyTorch is installed.

    python -m reduction_rdx_sum_gb300.build [--force] [-DNAME=VALUE ...]
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "librdx.so")
MARSHAL = os.path.join(PKG, "_marshal.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                     "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build librdx.so")
    return cand


def _cuda_lib_dir(nvcc: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs() -> list[str]:
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _torch_dir() -> str | None:
    """PyTorch's folder; None without PyTorch, or with one that has no CUDA."""
    spec = importlib.util.find_spec("torch")
    path = spec.submodule_search_locations[0] if spec is not None else ""
    return path if os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


def torch_version() -> str:
    """The installed PyTorch's version, read without importing it."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return re.search(r"^__version__ = ['\"](.+)['\"]", f.read(), re.M).group(1)


def build_marshal(force: bool = False) -> str:
    """Compile the marshalling extension module; returns its path.  It is bound to the PyTorch and the Python that it was
    compiled for, which a note in _build/ names: for others it is compiled again."""
    torch_dir = _torch_dir()
    if torch_dir is None:
        raise RuntimeError("the marshalling module needs PyTorch with CUDA, which is not installed")
    src, note = os.path.join(CSRC, "marshal.cpp"), os.path.join(BUILD, "marshal.txt")
    fits = f"PyTorch {torch_version()} in {torch_dir}, Python {sys.version}"
    inputs = [src, os.path.join(INCLUDE, "rdx.h"), os.path.abspath(__file__)]
    if not force and os.path.exists(MARSHAL) and all(os.path.getmtime(p) <= os.path.getmtime(MARSHAL) for p in inputs):
        if os.path.exists(note) and open(note).read() == fits:
            return MARSHAL
    include = os.path.join(torch_dir, "include")
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DRDX_TORCH_VERSION="{torch_version()}"', "-I", INCLUDE, "-isystem", include,
           "-isystem", os.path.join(include, "torch", "csrc", "api", "include"), "-I", sysconfig.get_path("include"),
           "-I", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include"), src, "-o", tmp,
           "-L", os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on marshal.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    os.makedirs(BUILD, exist_ok=True)
    with open(note, "w") as f:
        f.write(fits)
    return MARSHAL


def build(force: bool = False, defines: list[str] | None = None, out: str = LIB, verbose: bool = False) -> str:
    """Compile and link librdx.so; returns its path.  The in-tree library's marshalling module, too, where PyTorch is
    installed: C programs need neither."""
    if out != LIB or _torch_dir() is None:
        return _build_library(force, defines, out, verbose)
    with ThreadPoolExecutor(1) as ex:
        marshal = ex.submit(build_marshal, force)
        path = _build_library(force, defines, out, verbose)
        marshal.result()
    return path


def _build_library(force: bool, defines: list[str] | None, out: str, verbose: bool) -> str:
    if not force and not defines and out == LIB and up_to_date(out):
        return out
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    extra = list(defines or [])

    def compile_one(src: str):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + f".{os.getpid()}.o")
        cmd = [nvcc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    srcs = sources()
    with ThreadPoolExecutor(len(srcs)) as ex:
        results = list(ex.map(compile_one, srcs))
    objs = [o for o, _ in results]
    with open(os.path.join(BUILD, "ptxas.txt"), "w") as f:
        for src, (_, log) in zip(srcs, results):
            f.write(f"== {os.path.basename(src)}\n{log}\n")
    tmp = out + f".tmp{os.getpid()}"
    libdir = _cuda_lib_dir(nvcc)
    cmd = [nvcc, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs,
           f"-L{libdir}", f"-Xlinker=-rpath,{libdir}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    for o in objs:
        os.remove(o)
    if verbose:
        print(f"built {out}")
    return out


if __name__ == "__main__":
    args = sys.argv[1:]
    defines = [a for a in args if a.startswith("-D")]
    outs = [a.split("=", 1)[1] for a in args if a.startswith("--out=")]
    if defines and not outs:
        raise SystemExit("a build with -D defines needs --out=PATH (the in-tree librdx.so is the default build)")
    build(force="--force" in args, defines=defines, out=outs[0] if outs else LIB, verbose=True)
