"""Builds the in-tree shared library ``libtcl_gb300.so`` from ``csrc/*.cu`` with nvcc, and where
PyTorch is installed the binding's own module (``tensors_path``) from ``csrc/tensors.cpp``. Where that module
cannot be compiled, a warning says why: the library needs neither PyTorch nor Python, and the binding's
calls go without it, in more of the host's time.

Every translation unit is compiled for sm_103a only
(``-gencode arch=compute_103a,code=sm_103a``), in parallel, into
``_build/``; the objects are linked with the static CUDA runtime into one
position-independent shared library next to this file. Rebuilds only what is
older than its sources or any header.
"""
from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB_NAME = "libtcl_gb300.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")
    return path


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def tensors_path() -> str:
    """Where the binding's own module for this Python and this PyTorch is. It is compiled against their classes'
    layouts, so that one compiled against others must never be loaded: each has a file of its own."""
    import torch
    of = (sysconfig.get_config_var("EXT_SUFFIX"), torch.__version__, torch.version.git_version, torch.version.cuda,
          int(torch._C._GLIBCXX_USE_CXX11_ABI))
    return os.path.join(PKG, f"_tensors-{hashlib.sha256(repr(of).encode()).hexdigest()[:12]}.so")


def _build_tensors(force: bool) -> str:
    """The module that asks PyTorch's tensors for their addresses (the library itself needs no PyTorch)."""
    try:
        import torch
    except ImportError:
        return ""
    if torch.version.cuda is None:   # (a PyTorch without GPUs: it has no tensors for the calls)
        return ""
    path = tensors_path()
    src = os.path.join(CSRC, "tensors.cpp")
    if not force and not _stale(path, [src, __file__, *glob.glob(os.path.join(INCLUDE, "*.h"))]):
        return ""
    tmp = path + f".tmp{os.getpid()}"
    home = os.path.dirname(torch.__file__)
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", os.path.join(home, "include"),
           "-isystem", os.path.join(home, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           "-I", sysconfig.get_path("include"), "-I", INCLUDE, src, "-o", tmp, "-L", os.path.join(home, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {os.path.basename(src)}:\n{r.stderr}")
    os.replace(tmp, path)
    return r.stderr


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = _headers()
    objs, todo = [], []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers + [__file__]):
            todo.append((src, obj))

    def compile_one(item):
        src, obj = item
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        return r.stderr

    with ThreadPoolExecutor(max_workers=jobs or min(len(todo) + 1, os.cpu_count() or 4)) as ex:
        tensors = ex.submit(_build_tensors, force)
        for log in ex.map(compile_one, todo):
            if verbose and log:
                print(log)
    if force or todo or _stale(LIB_PATH, objs):
        tmp = LIB_PATH + f".tmp{os.getpid()}"
        cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr}")
        os.replace(tmp, LIB_PATH)
    try:
        tensors.result()
    except (OSError, RuntimeError) as e:   # (no compiler for the host, no headers of Python, another PyTorch)
        warnings.warn(f"the binding's module was not built, its calls take some 15 us more of the host's time: {e}", RuntimeWarning,
                      stacklevel=2)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
