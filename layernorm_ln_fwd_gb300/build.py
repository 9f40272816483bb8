"""Build ``libln.so`` in-tree with nvcc for sm_103a (GB300).

Each ``csrc/*.cu`` file is compiled to an object in parallel, then the objects are linked
into ``layernorm_ln_fwd_gb300/libln.so`` (CUDA runtime linked statically).  Register and
shared-memory usage reported by ptxas is kept in ``_build/ptxas.log``.  Beside it ``csrc/binding.cpp``
becomes the extension module ``_binding_*.so`` of the torch and Python that are here (g++, torch's headers).  The
library needs neither; without the module the Python binding makes the same calls through ctypes.

Usage: ``python -m layernorm_ln_fwd_gb300.build [--force]``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libln.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
                     "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libln.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + [os.path.join(CSRC, "binding.cpp")] + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(
        glob.glob(os.path.join(CSRC, "*.h"))) + [os.path.join(INCLUDE, "ln.h"), __file__]


def binding_path() -> str | None:
    """Where the extension module for the torch and the Python that are here belongs, or None without a torch.  Its
    name has both versions: a module built against others is not this one."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    with open(os.path.join(os.path.dirname(spec.origin), "version.py")) as f:
        version = re.search(r"^__version__ = ['\"](.+)['\"]", f.read(), re.M).group(1)
    return os.path.join(PKG, "_binding_" + re.sub(r"\W", "_", f"{version}_{sys.implementation.cache_tag}") + ".so")


def _built() -> list:
    """What a build makes here: the library, and the extension module where it can be built."""
    binding = binding_path() if shutil.which("g++") else None
    return [LIB] + ([binding] if binding else [])


def up_to_date() -> bool:
    made = _built()
    if not all(os.path.exists(m) for m in made):
        return False
    t = min(os.path.getmtime(m) for m in made)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _compile(src: str) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src).replace(".cu", ".o"))
    cmd = [nvcc()] + NVCC_FLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_binding(path: str) -> str:
    """The extension module, against the torch that is here; returns its temporary name."""
    import sysconfig

    import torch
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "binding.cpp"), "-o", tmp, "-L", libs, f"-Wl,-rpath,{libs}", "-ltorch_python",
           "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    return tmp


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    binding = (_built() + [None])[1]
    with cf.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        module = ex.submit(_compile_binding, binding) if binding else None
        results = list(ex.map(_compile, srcs))
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for (obj, log) in results:
            f.write(f"==== {os.path.basename(obj)}\n{log}\n")
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc()] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if module:  # (whatever comes of it, the library is there)
        os.replace(module.result(), binding)
    if verbose:
        print(f"built {LIB}" + ("" if module else " (no g++ or no torch: without the extension module)"))
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True)
