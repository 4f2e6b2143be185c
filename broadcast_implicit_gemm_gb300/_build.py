"""Compile the CUDA library (csrc/*.cu) into libbigemm.so, in place, for sm_103a.

Each translation unit is compiled by nvcc in parallel; the objects are linked
into one shared library next to this file, and layer_py.c and layer_tensor.cpp
are compiled into the extension module _layer.so beside it.  Rebuilds only when
a source or a header is newer than the libraries, or the module was built against
another torch or Python than the present ones, whose tensors it reads in place.

The library needs neither: where there is no torch with CUDA the module, whose calls
take its tensors, is left out.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import runpy
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libbigemm.so")
MODULE = os.path.join(HERE, "_layer.so")
STAMP = os.path.join(BUILD, "layer_for")     # what the module was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
         "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libbigemm.so")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(CSRC, "*.c")) + glob.glob(os.path.join(CSRC, "*.cpp"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def layer_name(version: str, git: str) -> str:
    """What a module is built for: a torch and a Python."""
    return f"torch {version} {git} {sysconfig.get_config_var('SOABI')}"


def _torch_root() -> str | None:
    """Where a torch with CUDA and its C++ headers is; None if there is none.  It is not imported."""
    spec = importlib.util.find_spec("torch")
    for root in (spec.submodule_search_locations if spec else None) or []:
        if all(os.path.exists(os.path.join(root, f)) for f in ("version.py", "lib/libc10_cuda.so",
                                                               "include/torch/csrc/autograd/python_variable.h")):
            return root
    return None


def layer_target() -> str | None:
    root = _torch_root()
    if root is None:
        return None
    v = runpy.run_path(os.path.join(root, "version.py"))
    return layer_name(v["__version__"], v["git_version"])


def _newer(path: str) -> bool:
    """Whether a file is there and no source is younger."""
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in _deps())


def _module_up_to_date() -> bool:
    target = layer_target()
    if target is None:
        return True
    if not _newer(MODULE) or not os.path.exists(STAMP):
        return False
    with open(STAMP) as f:
        return f.read() == target


def up_to_date() -> bool:
    return _newer(LIB) and _module_up_to_date()


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
    cmd = [nvcc(), *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
    if verbose and r.stderr:
        sys.stderr.write(r.stderr)
    return obj


def _run(cmd: list[str], what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {what}:\n{r.stderr}")


def _build_module() -> None:
    root, target = _torch_root(), layer_target()
    if root is None:
        return
    cc, cxx = shutil.which("gcc") or shutil.which("cc"), shutil.which("g++") or shutil.which("c++")
    if not cc or not cxx:
        raise RuntimeError("no C and C++ compiler found: gcc and g++ are required to build _layer.so")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = MODULE + f".tmp{os.getpid()}"
    objs = [os.path.join(BUILD, n) for n in ("layer_py.o", "layer_tensor.o")]
    common = ["-O2", "-fPIC", "-Wall", "-I", INCLUDE, "-I", CSRC, "-I", sysconfig.get_paths()["include"]]
    _run([cc, "-std=c11", *common, f'-DLAYER_BUILT_FOR="{target}"', "-c", os.path.join(CSRC, "layer_py.c"), "-o", objs[0]],
         "layer_py.c")
    # (torch's own headers, whose warnings are not ours)
    _run([cxx, "-std=c++17", *common, "-isystem", os.path.join(root, "include"), "-isystem",
          os.path.join(root, "include", "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"), "-c",
          os.path.join(CSRC, "layer_tensor.cpp"), "-o", objs[1]], "layer_tensor.cpp")
    # torch has loaded its libraries by the time this one is
    _run([cxx, "-shared", *objs, "-o", tmp, "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
          "-lc10"], "_layer.so")
    os.replace(tmp, MODULE)
    with open(STAMP + f".tmp{os.getpid()}", "w") as f:
        f.write(target)
    os.replace(STAMP + f".tmp{os.getpid()}", STAMP)


def _build_library(verbose: bool, jobs: int | None) -> None:
    srcs = sources()
    jobs = jobs or min(len(srcs), max(2, os.cpu_count() or 2))
    with cf.ThreadPoolExecutor(jobs) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(1) as ex:
        # beside the library, which does not wait for it
        module = ex.submit(_build_module) if force or not _module_up_to_date() else None
        if force or not _newer(LIB):
            _build_library(verbose, jobs)
        if module:
            module.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
