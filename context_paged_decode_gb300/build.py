"""Build libdcp.so (sm_103a) in-tree with nvcc: one object per .cu, compiled
in parallel, then linked into a shared library next to this file; and with the
host compiler the extension that hands tensors to it (_binding.so)."""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libdcp.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _sources(d):
    return sorted(os.path.join(d, f) for f in os.listdir(d) if f.endswith(".cu"))


def _headers(d):
    return [os.path.join(d, f) for f in os.listdir(d) if f.endswith((".cuh", ".h"))]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _compile(src, obj, extra=()):
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr}")
    return r.stderr


def build_library(lib=LIB, srcdir=CSRC, name="dcp", verbose=False, extra=()) -> str:
    """Compile and link one shared library from the .cu files of srcdir."""
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources(srcdir)
    deps = srcs + _headers(srcdir) + _headers(os.path.join(ROOT, "include")) + [__file__]
    if not _stale(lib, deps):
        return lib
    objs = [os.path.join(BUILD, f"{name}_{os.path.basename(s)[:-3]}.o") for s in srcs]
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs), os.cpu_count() or 4)) as ex:
        logs = list(ex.map(lambda so: _compile(so[0], so[1], extra), zip(srcs, objs)))
    if verbose:
        for s, log in zip(srcs, logs):
            if log.strip():
                print(os.path.basename(s), log, file=sys.stderr)
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *objs, "-lcudart_static", "-ldl", "-lrt",
           "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def build_binding() -> str:
    """Compile the Python extension (against this machine's torch and Python)."""
    src = os.path.join(HERE, "binding", "dcp_binding.cpp")
    out = os.path.join(HERE, "_binding.so")
    if not _stale(out, [src, __file__, *_headers(os.path.join(ROOT, "include"))]):
        return out
    import sysconfig

    import torch
    home = os.path.dirname(torch.__file__)
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        raise RuntimeError("g++ not found")
    inc = [os.path.join(home, "include"), os.path.join(ROOT, "include"),
           sysconfig.get_paths()["include"],
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")]
    libs = os.path.join(home, "lib")
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(f"-I{i}" for i in inc), src, "-o", out + ".tmp", f"-L{libs}", f"-Wl,-rpath,{libs}",
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-ldl"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx} failed for the binding:\n{r.stderr}")
    os.replace(out + ".tmp", out)
    return out


def build_all(verbose=False):
    synth_dir = os.path.join(ROOT, "workloads")
    with cf.ThreadPoolExecutor(max_workers=3) as ex:
        jobs = [ex.submit(build_library, verbose=verbose),
                ex.submit(build_library, os.path.join(synth_dir, "libdcp_synth.so"), synth_dir,
                          "synth", verbose=verbose),
                ex.submit(build_binding)]
        return [j.result() for j in jobs]


if __name__ == "__main__":
    for p in build_all(verbose="-v" in sys.argv):
        print(p)
