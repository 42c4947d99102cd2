"""Build libmoe_b200.so (sm_100a) in-tree with nvcc.

Each .cu under csrc/ compiles to an object in _build/; the objects link into
sparse_moe_layer_biased_b200/libmoe_b200.so with the CUDA runtime linked statically
(the library then loads on a host without a driver; it needs one only to run).
The debug variant (`--debug`) compiles the same sources with MOE_DEBUG into _build/debug/
and links libmoe_b200_debug.so: device-side range checks of every index read from device
data, reported through moe_check_device() as MOE_ERR_DEVICE_BOUNDS.
csrc/calls.cpp becomes the extension module _calls-torch<version>.<Python's ABI>.so beside them (g++, PyTorch's
headers), which TokenSorter alone needs: where it cannot be built, a warning says so and the library is there.
`python -m sparse_moe_layer_biased_b200.build [--force] [--debug] [--verbose-ptxas]`.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OBJ = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libmoe_b200.so")
LIB_DEBUG = os.path.join(PKG, "libmoe_b200_debug.so")
INCLUDE = os.path.join(ROOT, "include")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(f) for f in files)


def _compile(src, verbose_ptxas, debug=False):
    obj = os.path.join(OBJ, "debug" if debug else "", os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, *(["-DMOE_DEBUG"] if debug else []), "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def calls_path() -> str:
    """Where the extension module for this PyTorch and Python is: one built for others is not loaded by them."""
    import torch

    return os.path.join(PKG, f"_calls-torch{torch.__version__}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_calls(force: bool = False) -> str:
    """The extension module of TokenSorter's calls. It uses libmoe_b200.so by addresses that it is given."""
    src, out = os.path.join(CSRC, "calls.cpp"), calls_path()
    fresh = os.path.exists(out) and os.path.getmtime(out) >= _deps()
    if fresh and not force:
        return out
    if not fresh and os.path.exists(out):
        os.remove(out)  # not to be loaded with a newer library, should the build fail
    import torch

    base = os.path.dirname(torch.__file__)
    libs = os.path.join(base, "lib")
    tmp = out + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"), src, "-o", tmp,
           "-L", libs, f"-Wl,-rpath,{libs}", "-lc10", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose_ptxas: bool = False, debug: bool = False) -> str:
    lib = build_library(force, verbose_ptxas, debug)
    try:
        build_calls(force)
    except (OSError, RuntimeError) as e:
        warnings.warn(f"TokenSorter's extension module is not built, all else is: {e}", RuntimeWarning, stacklevel=2)
    return lib


def build_library(force: bool = False, verbose_ptxas: bool = False, debug: bool = False) -> str:
    lib = LIB_DEBUG if debug else LIB
    if not force and os.path.exists(lib) and os.path.getmtime(lib) >= _deps():
        return lib
    os.makedirs(os.path.join(OBJ, "debug") if debug else OBJ, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose_ptxas, debug), sources()))
    if verbose_ptxas:
        for obj, log in results:
            print(f"== {os.path.basename(obj)}\n{log}", file=sys.stderr)
    objs = [o for o, _ in results]
    tmp = lib + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--verbose-ptxas" in sys.argv,
                debug="--debug" in sys.argv))
