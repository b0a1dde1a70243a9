"""Build the CUDA library in-tree with nvcc for sm_100a.

It also compiles binding/fast.cpp with g++ against PyTorch's headers into an extension
module, _fast (the paged operators' calls without the interpreter), which links the
library. Without PyTorch, or where that fails, the library is complete without it: the
Python binding makes every call itself.

The shared library statically links the CUDA runtime and exports only the
``cmp_*`` entry points declared in include/cmp.h, so it can be loaded next to
any other CUDA runtime (for example PyTorch's) without symbol clashes.
"""

from __future__ import annotations

import concurrent.futures
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libcmp_b200.so")
FAST_SRC = os.path.join(PKG, "binding", "fast.cpp")
FAST = os.path.join(PKG, "_fast" + sysconfig.get_config_var("EXT_SUFFIX"))  # names the Python it is for
FAST_KEY = os.path.join(OBJDIR, "fast.key")  # the PyTorch and Python it was built with
# measurement build: the same sources with the decode kernel's phase stamps
# (-DCMP_PHASE_STAMPS), for bench.py --only decode-phases
PHASES_OBJDIR = os.path.join(PKG, "_build", "phases")
PHASES_LIB = os.path.join(PKG, "libcmp_b200_phases.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
                 "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    nvcc = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    return nvcc


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max([os.path.getmtime(h) for h in hs] + [0.0])


def _compile(src: str, obj: str, extra: list, verbose: bool) -> None:
    cmd = [_nvcc(), *CFLAGS, *extra, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)


def build(verbose: bool = False, force: bool = False, ptxas_info: bool = False,
          phases: bool = False) -> str:
    """Compile every csrc/*.cu and link libcmp_b200.so (with phases=True the
    phase-stamp measurement build, libcmp_b200_phases.so). Returns the library path."""
    objdir, lib = (PHASES_OBJDIR, PHASES_LIB) if phases else (OBJDIR, LIB)
    os.makedirs(objdir, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr = _newest_header()
    extra = (["-Xptxas", "-v"] if ptxas_info else []) + (["-DCMP_PHASE_STAMPS"] if phases else [])
    jobs = []
    for s in srcs:
        o = os.path.join(objdir, os.path.basename(s)[:-3] + ".o")
        if force or ptxas_info or not os.path.exists(o) or \
                os.path.getmtime(o) < max(os.path.getmtime(s), hdr):
            jobs.append((s, o))
    if jobs:
        with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(jobs))) as ex:
            list(ex.map(lambda so: _compile(so[0], so[1], extra, verbose or ptxas_info), jobs))
    objs = [os.path.join(objdir, os.path.basename(s)[:-3] + ".o") for s in srcs]
    if jobs or force or not os.path.exists(lib):
        cmd = [_nvcc(), *ARCH, "-shared", "-o", lib, *objs, "-cudart", "static",
               "-Xlinker", "--exclude-libs,ALL", "-Xlinker", "-Bsymbolic", "-lrt", "-ldl",
               "-lpthread"]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    if not phases:
        build_fast(verbose, force)
    return lib


def build_fast(verbose: bool = False, force: bool = False):
    """Compile binding/fast.cpp against PyTorch's headers. Returns the module's path, or
    None (with a warning, unless there is no PyTorch) if it could not be built."""
    spec = importlib.util.find_spec("torch")  # without importing it
    if spec is None:
        return None
    torch = spec.submodule_search_locations[0]
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        warnings.warn("the compiled binding was not built: PyTorch does not say its version")
        return None
    key = f"{version}\n{torch}\n{sys.version}\n"
    newest = max(os.path.getmtime(f) for f in [FAST_SRC, __file__] + glob.glob(os.path.join(INCLUDE, "*.h")))
    if not force and os.path.exists(FAST) and os.path.getmtime(FAST) >= newest and os.path.exists(FAST_KEY):
        with open(FAST_KEY) as f:
            if f.read() == key:
                return FAST
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    libs = os.path.join(torch, "lib")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DFAST_TORCH_VERSION="{version}"', "-I", INCLUDE, "-isystem", os.path.join(torch, "include"),
           "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           FAST_SRC, "-o", FAST, "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
           "-L", PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    if verbose:
        print(" ".join(cmd), flush=True)
    if os.path.exists(FAST):  # never one that is older than what it was built from
        os.remove(FAST)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        warnings.warn(f"the compiled binding was not built: g++ failed for fast.cpp:\n{r.stdout}\n{r.stderr}")
        return None
    os.makedirs(OBJDIR, exist_ok=True)
    with open(FAST_KEY, "w") as f:
        f.write(key)
    return FAST


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv,
                ptxas_info="--ptxas" in sys.argv, phases="--phases" in sys.argv))
