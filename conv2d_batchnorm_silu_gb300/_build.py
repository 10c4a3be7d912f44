"""Builds the in-tree CUDA library ``libconvbnsilu.so`` for sm_103a with nvcc.

One object per translation unit, compiled in parallel, then linked into a
shared library with the CUDA runtime linked statically; beside it, with g++,
``_token_ops.so``, the Python calls of the token-wise operators over PyTorch's
C++ tensors, where PyTorch is installed.  Each is rebuilt only when a source or
header of its own is newer, the second also for another PyTorch or Python.
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libconvbnsilu.so")
BINDING_SOURCE = os.path.join(CSRC, "binding.cpp")
BINDING_PATH = os.path.join(PKG_DIR, "_token_ops.so")
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return path


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers() -> list[str]:
    return glob.glob(os.path.join(ROOT, "include", "*.h"))


def _newer_than(path: str, inputs: list[str]) -> bool:
    """Whether `path` exists and none of its inputs has changed since."""
    return os.path.exists(path) and all(os.path.getmtime(f) <= os.path.getmtime(path) for f in inputs)


def _library_up_to_date() -> bool:
    return _newer_than(LIB_PATH, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                       + _headers() + [os.path.abspath(__file__)])


def _torch_dir() -> str | None:
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec and spec.submodule_search_locations else None


def _built_for() -> str:
    """The PyTorch and the Python that the binding is compiled against."""
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # not installed as a package
        torch = _torch_dir()
    return f"torch {torch}, {sys.implementation.cache_tag}"


def _stamp_path() -> str:
    return os.path.join(BUILD_DIR, "binding.for")


def _binding_up_to_date() -> bool:
    if not _newer_than(BINDING_PATH, _headers() + [BINDING_SOURCE, os.path.abspath(__file__)]):
        return False
    try:
        with open(_stamp_path()) as f:
            return f.read() == _built_for()
    except FileNotFoundError:
        return False


def up_to_date() -> bool:
    return _library_up_to_date() and (_torch_dir() is None or _binding_up_to_date())


def _compile_binding() -> str:
    """The binding's object file."""
    torch_include = os.path.join(_torch_dir(), "include")
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    obj = os.path.join(BUILD_DIR, "binding.o")
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-I", sysconfig.get_paths()["include"],
           "-I", torch_include, "-I", os.path.join(torch_include, "torch", "csrc", "api", "include"),
           "-I", cuda_include, "-I", os.path.join(ROOT, "include"), "-c", BINDING_SOURCE, "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SOURCE}:\n{res.stdout}\n{res.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    tmp = BINDING_PATH + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "c++", "-shared", "-o", tmp, obj, "-L", PKG_DIR, "-lconvbnsilu",
           "-Wl,-rpath,$ORIGIN", "-L", os.path.join(_torch_dir(), "lib"), "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
           "-lc10_cuda", "-lc10"]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, BINDING_PATH)
    with open(_stamp_path(), "w") as f:
        f.write(_built_for())


def build(force: bool = False, verbose: bool = False, extra_flags: list[str] | None = None) -> str:
    """Compile every ``csrc/*.cu`` for sm_103a and link ``libconvbnsilu.so``, and the binding beside it where PyTorch
    is installed; returns the library's path.  The library is in place before an error of the binding's is raised."""
    library = force or not _library_up_to_date()
    with_binding = _torch_dir() is not None and (force or not _binding_up_to_date())
    if not library and not with_binding:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    flags = NVCC_FLAGS + ARCH_FLAGS + (extra_flags or [])

    def compile_one(src: str) -> str:
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc(), *flags, "-c", src, "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{res.stdout}\n{res.stderr}")
        if verbose and (res.stdout or res.stderr):
            print(res.stdout + res.stderr)
        return obj

    srcs = sources() if library else []
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        binding = ex.submit(_compile_binding) if with_binding else None
        objs = list(ex.map(compile_one, srcs))
    if library:
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH_FLAGS, "-shared", "-cudart", "static", "-o", tmp, *objs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"link failed:\n{res.stdout}\n{res.stderr}")
        os.replace(tmp, LIB_PATH)
    if binding is not None:
        _link_binding(binding.result())
    return LIB_PATH
