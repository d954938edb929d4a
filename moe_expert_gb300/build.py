"""Builds libmoex.so (the C-ABI library) in the package directory with nvcc,
and the Python extension module over it with the host compiler.

Every .cu under csrc/ is compiled for sm_103a only, in parallel, then linked
into one shared library.  csrc/binding.cpp is compiled beside them against
Python's and torch's headers into _native.so, which links to libmoex.so; where
there is no torch, the library alone is built, and a message says so.
Objects go to moe_expert_gb300/_build/.  Run as
``python -m moe_expert_gb300.build`` or call ``build()``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoex.so")
NATIVE = os.path.join(PKG, "_native.so")
BINDING = os.path.join(CSRC, "binding.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    cand = [os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"]
    for c in cand:
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers_digest() -> str:
    h = hashlib.sha256()
    for p in sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                    + glob.glob(os.path.join(PKG, "..", "include", "*.h"))):
        with open(p, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def _compile(src: str, extra) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def _torch_dir():
    spec = importlib.util.find_spec("torch")  # without the cost of importing it
    if spec is None or not spec.submodule_search_locations:
        return None
    return list(spec.submodule_search_locations)[0]


def _compile_binding() -> str:
    obj = os.path.join(BUILD, "binding.cpp.o")
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-w", "-I" + sysconfig.get_paths()["include"],
           "-I" + inc, "-I" + os.path.join(inc, "torch", "csrc", "api", "include"), "-I" + cuda, "-c", BINDING,
           "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {BINDING}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding() -> None:
    lib = os.path.join(_torch_dir(), "lib")
    tmp = NATIVE + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, os.path.join(BUILD, "binding.cpp.o"), "-L" + PKG,
           "-l:libmoex.so", "-Wl,-rpath,$ORIGIN", "-L" + lib, "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of the Python binding failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)


def build(verbose: bool = False, extra=()) -> str:
    """Compiles every source, links libmoex.so and (with torch) the extension module; returns the library's path."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    digest = _headers_digest()
    stamp = os.path.join(BUILD, "headers.sha")
    old = open(stamp).read() if os.path.exists(stamp) else ""
    todo = []
    for s in srcs:
        obj = os.path.join(BUILD, os.path.basename(s) + ".o")
        if old != digest or not os.path.exists(obj) or os.path.getmtime(obj) < os.path.getmtime(s):
            todo.append(s)
    jobs = [lambda s=s: _compile(s, list(extra)) for s in todo]
    bobj = os.path.join(BUILD, "binding.cpp.o")
    binding = _torch_dir() is not None
    if not binding:
        sys.stderr.write("torch not found: libmoex.so is built without the Python binding _native.so\n")
        for p in (bobj, NATIVE):  # of another build of the library
            if os.path.exists(p):
                os.remove(p)
    elif old != digest or not os.path.exists(bobj) or os.path.getmtime(bobj) < os.path.getmtime(BINDING):
        jobs.append(_compile_binding)
    if jobs:
        with cf.ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
            list(ex.map(lambda j: j(), jobs))
    objs = [os.path.join(BUILD, os.path.basename(s) + ".o") for s in srcs]
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if binding:
        _link_binding()
    with open(stamp, "w") as f:
        f.write(digest)
    if verbose:
        print(LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True, extra=sys.argv[1:])
