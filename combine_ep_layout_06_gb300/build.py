"""Build libep_gb300.so in-tree with nvcc for sm_103a (no cmake), and
_moe.so, the Python binding of the routing, loss and product calls.

Each .cu file under csrc/ compiles to an object in parallel, then nvcc links
one shared library with the CUDA runtime linked statically, so that loading
it needs only the driver, and building it only nvcc.  The binding is one C++
file against torch's headers, compiled next to them and linked to that library;
without torch, which alone could load it, it is left out.  Usage: ``python -m
combine_ep_layout_06_gb300.build [--ptxas-verbose]``.
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
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libep_gb300.so")
BINDING_SRC = os.path.join(CSRC, "moe_binding.cpp")
BINDING = os.path.join(BUILD, "_moe.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-O2", f"-I{os.path.join(ROOT, 'include')}",
              *ARCH]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build "
                       "libep_gb300.so")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [
        os.path.join(ROOT, "include", "ep_api.h"), os.path.abspath(__file__)]


def library_up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _binding_made_for() -> str:
    """What a binding fits besides its sources: one torch, one Python."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}\n"


def binding_up_to_date() -> bool:
    """Newer than its source, than the structs it shares with the library and
    than this file, and made for the torch and the Python that run."""
    try:
        with open(BINDING + ".for") as f:
            made_for = f.read()
        t = os.path.getmtime(BINDING)
    except OSError:
        return False
    deps = [BINDING_SRC, os.path.join(ROOT, "include", "ep_api.h"), os.path.abspath(__file__)]
    return made_for == _binding_made_for() and all(os.path.getmtime(d) <= t for d in deps)


def _has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r.stderr


def _torch_dir() -> str:
    import torch
    return os.path.dirname(os.path.abspath(torch.__file__))


def _compile_binding() -> str:
    import torch
    cxx = shutil.which("g++")
    if not cxx:
        raise RuntimeError("g++ not found: it is required to build the Python binding")
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    obj = os.path.join(BUILD, "moe_binding.o")
    _run([cxx, "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
          "-isystem", sysconfig.get_paths()["include"], "-isystem", cuda, "-c", BINDING_SRC, "-o", obj],
         f"g++ failed on {BINDING_SRC}")
    return obj


def _link_binding(obj: str):
    tmp = BINDING + f".{os.getpid()}.tmp"
    _run([shutil.which("g++"), "-shared", "-o", tmp, obj, f"-L{os.path.join(_torch_dir(), 'lib')}", "-ltorch_python",
          "-ltorch_cpu", "-lc10_cuda", "-lc10", f"-L{BUILD}", "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"],
         "link of the Python binding failed")
    os.replace(tmp, BINDING)
    with open(BINDING + ".for", "w") as f:
        f.write(_binding_made_for())


def build_library(force: bool = False, ptxas_verbose: bool = False) -> str:
    """EP_NVTX=1 in the environment compiles NVTX ranges around the entry
    points in (for timelines and ncu range filters); they are off otherwise."""
    if not force and not ptxas_verbose and library_up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    if os.environ.get("EP_NVTX", "0") not in ("", "0"):
        extra.append("-DEP_NVTX=1")

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        return obj, _run([nvcc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj], f"nvcc failed on {src}")

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(compile_one, sources()))
    if ptxas_verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".{os.getpid()}.tmp"
    _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *[o for o, _ in results]], "link failed")
    os.replace(tmp, LIB)
    return LIB


def build_binding(force: bool = False) -> str:
    """The binding, for a library that is there."""
    if force or not binding_up_to_date():
        _link_binding(_compile_binding())
    return BINDING


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    """Both, compiled side by side.  The library is in place before a binding
    that does not build is an error."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(_compile_binding) if _has_torch() and (force or not binding_up_to_date()) else None
        build_library(force, ptxas_verbose)
        if binding:
            _link_binding(binding.result())
    if not _has_torch():
        sys.stderr.write("torch is not installed: the Python binding is left out\n")
    return LIB


if __name__ == "__main__":
    print(build(force=True, ptxas_verbose="--ptxas-verbose" in sys.argv))
