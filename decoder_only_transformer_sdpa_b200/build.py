"""Build step of the CUDA library: compiles csrc/*.cu for sm_100a with nvcc
into ``libattn.so`` next to this file (in-tree, so it travels with the
repository).  Run ``python decoder_only_transformer_sdpa_b200/build.py``
(a plain script: it does not import the package, which needs the library).
``--debug`` builds ``libattn_debug.so`` instead: the same kernels with the
device-side bounds checks compiled in (-DATTN_DEVICE_CHECKS); select it with
the ATTN_LIBRARY environment variable.  ``_q8.so``, the Python module of the
8-bit cache's calls, is host code against torch's headers, built by g++ after
either; the library needs neither torch nor the module."""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libattn.so")
BUILD_DEBUG = os.path.join(HERE, "_build_debug")
LIB_DEBUG = os.path.join(HERE, "libattn_debug.so")
ROOT = os.path.dirname(HERE)

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = "g++"
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-fvisibility=hidden",
         f"-I{os.path.join(ROOT, 'include')}", "-Xptxas", "-warn-spills"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.h"))) + \
        sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [os.path.join(ROOT, "include", "attn.h")]


def _torch_version(folder: str) -> str:
    """The version that the torch installed there reports, by its version.py alone."""
    with open(os.path.join(folder, "version.py")) as f:
        return re.search(r"^__version__ = ['\"]([^'\"]+)['\"]", f.read(), re.M).group(1)


def build_binding(force: bool = False) -> Optional[str]:
    """The module _q8 (csrc/q8_binding.cpp); torch is found but not imported.
    None without torch, where nothing could call it.  The module carries the
    versions of torch and Python that it is built against, and is built anew for
    others."""
    src, so = os.path.join(CSRC, "q8_binding.cpp"), os.path.join(HERE, "_q8.so")
    deps = [src, os.path.join(ROOT, "include", "attn.h")]
    found = importlib.util.find_spec("torch")
    if found is None:
        sys.stderr.write(f"{so} is not built: it binds the 8-bit cache to torch, which is not installed\n")
        return None
    torch = found.submodule_search_locations[0]
    built_for = f"torch {_torch_version(torch)}, {sys.implementation.cache_tag}"
    if not force and os.path.exists(so) and all(os.path.getmtime(p) <= os.path.getmtime(so) for p in deps):
        with open(so, "rb") as f:
            if f"built for {built_for}\0".encode() in f.read():
                return so
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")]
    tmp = so + f".tmp{os.getpid()}"
    r = subprocess.run([CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
                        f'-DATTN_BUILT_FOR="{built_for}"', *(f"-I{d}" for d in include),
                        src, "-o", tmp, "-L" + os.path.join(torch, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
                        "-ltorch_python"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed on {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, so)
    return so


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src: str, verbose_ptxas: bool, debug: bool = False) -> str:
    obj = os.path.join(BUILD_DEBUG if debug else BUILD, os.path.basename(src) + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, *(["-DATTN_DEVICE_CHECKS"] if debug else []), "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose_ptxas and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False, debug: bool = False) -> str:
    lib = _build_library(force, verbose_ptxas, debug)
    build_binding(force)
    return lib


def _build_library(force: bool, verbose_ptxas: bool, debug: bool) -> str:
    lib = LIB_DEBUG if debug else LIB
    if not force and up_to_date(lib):
        return lib
    os.makedirs(BUILD_DEBUG if debug else BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose_ptxas, debug), _sources()))
    tmp = lib + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, *ARCH, "-shared", "-o", tmp, *objs])
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv, debug="--debug" in sys.argv))
