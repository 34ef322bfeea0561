"""Build libgemm_f16.so in-tree with nvcc for sm_103a.

    python -m dense_gemm_gb300.build [--force] [--debug]

--debug builds libgemm_f16_debug.so instead: the same kernels with device-side
bounds and alignment checks (GEMM_DEBUG) that report GEMM_ERR_CHECK instead of
trapping. The binding loads it when GEMM_LIBRARY=debug.

Two translation units, compiled side by side, one -gencode, static CUDA runtime; no cmake. The same
command works on x86-64 and aarch64 hosts. Beside it, the CPython extension
_native (ops.py's argument marshalling, on PyTorch's C++ API) is built with the
host compiler, at the same time. Its file's name carries the Python and PyTorch it
was built for, so that another's is never loaded. The library needs none of what that takes:
where this PyTorch has no CUDA parts, or there is no C++ compiler or no Python.h,
the library is built without it and ops.py's calls raise.
"""
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libgemm_f16.so")
DEBUG_LIB = os.path.join(HERE, "libgemm_f16_debug.so")
SOURCES = [os.path.join(CSRC, "library.cu"), os.path.join(CSRC, "ops_rows.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, f) for f in ("gemm_f16.cu", "ops.cu", "ops_block.cu", "gemm_kernel.cuh", "gemm_pair.cuh",
                                                     "elements.cuh", "ops_eight.cuh", "ops_linear.cuh", "ops_norm.cuh", "ops_rows.h", "rows_check.cuh",
                                                     "ptx.cuh")] + \
    [os.path.join(INCLUDE, f) for f in ("gemm_f16.h", "gemm_ops.h")]

NATIVE_DEPENDS = [os.path.join(CSRC, "native.cpp")] + [os.path.join(INCLUDE, f) for f in ("gemm_f16.h", "gemm_ops.h")]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def command(out: str, verbose_ptxas: bool = False, debug: bool = False):
    cmd = [nvcc(), *ARCH, "-t", str(len(SOURCES)), "-O3", "-lineinfo", "-std=c++17", "-shared", "-Xcompiler", "-fPIC",
           "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC, "-o", out, *SOURCES]
    if verbose_ptxas:
        cmd.insert(1, "-Xptxas=-v")
    if debug:
        cmd.insert(1, "-DGEMM_DEBUG")
    return cmd


def up_to_date(lib: str = LIB, depends=None) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in (DEPENDS if depends is None else depends))


def torch_dir() -> str:
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def native_path() -> str:
    """The extension's file for this Python and PyTorch, whose version is read, not imported."""
    with open(os.path.join(torch_dir(), "version.py")) as f:
        version = re.search(r"""__version__ = ['"]([^'"]+)['"]""", f.read()).group(1)
    return os.path.join(HERE, f"_native.{sysconfig.get_config_var('SOABI')}-torch{version}.so")


def cxx() -> str:
    return os.environ.get("CXX", "g++")


def native_unbuildable() -> str:
    """Why the extension cannot be built on this machine; empty where it can."""
    if shutil.which(cxx()) is None:
        return f"no C++ compiler ({cxx()})"
    needed = [os.path.join(torch_dir(), "include", "c10", "cuda", "CUDAStream.h"), os.path.join(torch_dir(), "lib", "libc10_cuda.so"),
              os.path.join(sysconfig.get_paths()["include"], "Python.h")]
    missing = [p for p in needed if not os.path.exists(p)]
    return f"{missing[0]} is missing" if missing else ""


def native_command(out: str):
    """The host compiler's command for the extension; found without importing torch
    (a slow import), which the extension's own process has loaded when it is used."""
    lib = os.path.join(torch_dir(), "lib")
    inc = [os.path.join(torch_dir(), "include"), os.path.join(torch_dir(), "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"), INCLUDE, sysconfig.get_paths()["include"]]
    return [cxx(), "-O2", "-std=c++17", "-Wall", "-shared", "-fPIC", "-fvisibility=hidden",
            *(f"-I{d}" for d in inc), "-o", out, NATIVE_DEPENDS[0], f"-L{lib}", f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch",
            "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build_native(force: bool = False) -> str:
    native = native_path()
    if not force and up_to_date(native, NATIVE_DEPENDS):
        return native
    tmp = native + f".tmp{os.getpid()}"
    subprocess.run(native_command(tmp), check=True)
    os.replace(tmp, native)
    return native


def build(force: bool = False, verbose_ptxas: bool = False, debug: bool = False) -> str:
    lib = DEBUG_LIB if debug else LIB
    with ThreadPoolExecutor(1) as beside:
        why = native_unbuildable()
        native = None if why else beside.submit(build_native, force)
        if why:
            print(f"{os.path.basename(native_path())} is not built: {why} (the operators of ops.py will raise)", file=sys.stderr)
        if force or not up_to_date(lib):
            tmp = lib + f".tmp{os.getpid()}"
            subprocess.run(command(tmp, verbose_ptxas, debug), check=True)
            os.replace(tmp, lib)
        if native is not None:
            native.result()
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv, debug="--debug" in sys.argv))
