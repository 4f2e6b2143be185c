"""Compile the CUDA library (csrc/*.cu) into libbigemm.so, in place, for sm_103a.

Each translation unit is compiled by nvcc in parallel; the objects are linked
into one shared library next to this file, and layer_py.c and layer_tensor.cpp
are compiled into the extension module _layer.so beside it.  Rebuilds only when
a source or a header is newer than the libraries.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
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


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MODULE):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(MODULE))
    return all(os.path.getmtime(d) <= t for d in _deps())


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
    cc, cxx = shutil.which("gcc") or shutil.which("cc"), shutil.which("g++") or shutil.which("c++")
    if not cc or not cxx:
        raise RuntimeError("no C and C++ compiler found: gcc and g++ are required to build _layer.so")
    torch = importlib.util.find_spec("torch").submodule_search_locations[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = MODULE + f".tmp{os.getpid()}"
    objs = [os.path.join(BUILD, n) for n in ("layer_py.o", "layer_tensor.o")]
    common = ["-O2", "-fPIC", "-Wall", "-I", INCLUDE, "-I", CSRC, "-I", sysconfig.get_paths()["include"]]
    _run([cc, "-std=c11", *common, "-c", os.path.join(CSRC, "layer_py.c"), "-o", objs[0]], "layer_py.c")
    # (torch's own headers, whose warnings are not ours)
    _run([cxx, "-std=c++17", *common, "-isystem", os.path.join(torch, "include"), "-isystem",
          os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-isystem", os.path.join(cuda, "include"), "-c",
          os.path.join(CSRC, "layer_tensor.cpp"), "-o", objs[1]], "layer_tensor.cpp")
    # torch has loaded its libraries by the time this one is
    _run([cxx, "-shared", *objs, "-o", tmp, "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10_cuda",
          "-lc10"], "_layer.so")
    os.replace(tmp, MODULE)


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs), max(2, os.cpu_count() or 2))
    with cf.ThreadPoolExecutor(jobs) as ex:
        module = ex.submit(_build_module)
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
        module.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lrt"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
