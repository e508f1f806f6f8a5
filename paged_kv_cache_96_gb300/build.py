"""Build the CUDA library in-tree: nvcc for sm_103a only.

    python -m paged_kv_cache_96_gb300.build

compiles every ``csrc/*.cu`` (device code, one ``-gencode`` each) and
``csrc/*.cpp`` (host-only runtime code) in parallel, CUDA runtime linked
statically, and links ``lib/libpaged_attention.so``; beside it the Python calls that
read torch tensors themselves (``pyext/calls.cpp``, host compiler and torch's headers).
Only the serving-step calls need those: where they do not compile the build warns, and
the calls raise when they are used.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
OBJDIR = os.path.join(HERE, "_build")
LIB = os.path.join(LIBDIR, "libpaged_attention.so")
CALLS_SRC = os.path.join(HERE, "pyext", "calls.cpp")
HEADER = os.path.join(os.path.dirname(HERE), "include", "paged_attention.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "--use_fast_math", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"),
                 "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build")


def _compile(src: str, verbose_ptxas: bool, objdir: str = OBJDIR, extra=()) -> str:
    obj = os.path.join(objdir, os.path.splitext(os.path.basename(src))[0] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas:
        sys.stderr.write(r.stderr)
    return obj


def calls_path(torch_version: str) -> str:
    """The extension for this Python and a version of torch, whose tensors' layout it
    is compiled for: both are part of its name, so that another's is never loaded."""
    return os.path.join(HERE, f"_calls.torch-{torch_version}" +
                        sysconfig.get_config_var("EXT_SUFFIX"))


def _build_calls() -> None:
    import torch
    calls = calls_path(torch.__version__)
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    tmp = calls + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(root, "include"),
           "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I" + cuda,
           CALLS_SRC, "-o", tmp, "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compiling {CALLS_SRC} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, calls)


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _newer(built: str, deps) -> bool:
    return os.path.exists(built) and \
        all(os.path.getmtime(d) <= os.path.getmtime(built) for d in deps)


def library_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [HEADER])


def calls_up_to_date() -> bool:
    import torch
    return _newer(calls_path(torch.__version__), [CALLS_SRC, HEADER])


def _build_library(lib: str, verbose_ptxas: bool, extra, objdir: str) -> None:
    os.makedirs(objdir, exist_ok=True)
    os.makedirs(os.path.dirname(lib), exist_ok=True)
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas, objdir, extra), srcs))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)


def build(force: bool = False, verbose_ptxas: bool = False, extra=(),
          out: str = None) -> str:
    """Compile and link; `extra` nvcc flags and `out` library path are for
    building tuning variants next to the default library."""
    lib = out or LIB

    def build_calls():
        if force or not calls_up_to_date():
            for stale in glob.glob(os.path.join(HERE, "_calls*.so")):
                with contextlib.suppress(FileNotFoundError):
                    os.remove(stale)  # of older sources, or for another torch or Python
            _build_calls()

    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        calls = ex.submit(build_calls) if out is None else None
        if force or out is not None or extra or not library_up_to_date():
            _build_library(lib, verbose_ptxas, extra,
                           OBJDIR if out is None else os.path.join(os.path.dirname(out), "_obj"))
        try:
            if calls is not None:
                calls.result()
        except Exception as e:
            warnings.warn(f"the serving-step calls were not built: {e}")
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
