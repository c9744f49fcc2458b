"""Builds libspecverify.so in-tree: every .cu under csrc/ compiled for
sm_103a (one -gencode, -lineinfo) in parallel, then linked with the static
CUDA runtime; and beside it _spec_torch.so, the cache calls' Python binding
(g++, against the installed PyTorch)."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIBDIR, "libspecverify.so")
BINDING = os.path.join(LIBDIR, "_spec_torch.so")
BINDING_SRC = os.path.join(CSRC, "spec_torch.cpp")
BINDING_FOR = os.path.join(LIBDIR, "_spec_torch.for")      # what the binding was built against
ROOT = os.path.dirname(HERE)

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libspecverify")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _built_for() -> str:
    """The binding uses PyTorch's and Python's C++ interfaces, which hold for one version."""
    import torch
    return f"torch {torch.__version__}, {sysconfig.get_config_var('SOABI')}"


def binding_up_to_date() -> bool:
    if not os.path.exists(BINDING) or not os.path.exists(BINDING_FOR):
        return False
    with open(BINDING_FOR) as f:
        if f.read() != _built_for():
            return False
    t = os.path.getmtime(BINDING)
    return all(os.path.getmtime(p) <= t for p in [BINDING_SRC] + glob.glob(os.path.join(ROOT, "include", "*.h")))


def build_binding() -> str:
    """Compile the cache calls' Python binding (no device code)."""
    import torch
    top = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I", os.path.join(top, "include"),
           "-I", os.path.join(top, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], "-I", os.path.join(cuda, "include"), BINDING_SRC, "-o", tmp,
           "-L", os.path.join(top, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cuda", "-lc10", "-lc10_cuda",
           "-L", os.path.join(cuda, "lib64"), "-lcudart"]
    os.makedirs(LIBDIR, exist_ok=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {BINDING_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(_built_for())
    return BINDING


def build(force: bool = False, verbose: bool = False, extra_flags=(), out: str = None) -> str:
    """Build the library (to `out` with `extra_flags` for a development
    variant, e.g. -DSPEC_TRACE; the default is the product library)."""
    lib = out or LIB
    with cf.ThreadPoolExecutor(max_workers=1) as one:
        stale = out is None and (force or not binding_up_to_date())
        binding = one.submit(build_binding) if stale else None     # beside the kernels' compilation
        lib = _build_library(force, verbose, extra_flags, lib, out)
        if binding is not None:
            binding.result()
    return lib


def _build_library(force, verbose, extra_flags, lib, out) -> str:
    if not force and out is None and up_to_date():
        return LIB
    objdir = os.path.join(os.path.dirname(lib), "obj" if out is None else "obj_" + os.path.basename(lib))
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout, r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force=True, verbose=True))
