"""Build libdfv.so in-tree: every .cu under csrc/ compiled for sm_103a only,
in parallel, then linked into one shared library (no cmake); and _dfvbind.so,
the Python binding's extension (host code, torch's headers), beside it."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdfv.so")
BIND = os.path.join(HERE, "_dfvbind.so")
BIND_SRC = os.path.join(CSRC, "binding.cpp")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-I", INCLUDE]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return [BIND_SRC] + _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + sorted(glob.glob(os.path.join(INCLUDE, "*.h")))


def _torch() -> str:
    """The torch that a binding built now is tied to."""
    try:
        import torch
    except ImportError:
        return ""
    return "%s %s\n" % (torch.__version__, os.path.dirname(torch.__file__))


def _stamp() -> str:
    return os.path.join(BUILD, "binding.torch")


def up_to_date() -> bool:
    if not all(os.path.exists(f) for f in (LIB, BIND, _stamp())):
        return False
    with open(_stamp()) as f:
        if f.read() != _torch():
            return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(BIND))
    return all(os.path.getmtime(f) <= t for f in _deps() + [__file__])


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [NVCC, *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
        if verbose and r.stderr:
            sys.stderr.write(r.stderr)
        return obj

    bind_obj = os.path.join(BUILD, "binding.o")

    def compile_binding():
        try:
            import torch
        except ImportError as e:
            raise RuntimeError("the binding needs torch's headers: %s" % e)
        at = os.path.join(os.path.dirname(torch.__file__), "include")
        cuda = os.path.join(os.path.dirname(os.path.dirname(shutil.which(NVCC) or "/usr/local/cuda/bin/nvcc")), "include")
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-I", sysconfig.get_paths()["include"], "-I", at,
               "-I", os.path.join(at, "torch", "csrc", "api", "include"), "-I", cuda, "-c", BIND_SRC, "-o", bind_obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("compiling the binding failed:\n%s\n%s" % (" ".join(cmd), r.stderr))

    with cf.ThreadPoolExecutor(max_workers=min(9, len(srcs) + 1)) as ex:
        binding = ex.submit(compile_binding)
        objs = list(ex.map(compile_one, srcs))
    # the C library needs nothing of torch and is linked whatever becomes of the binding
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, LIB)
    binding.result()
    import torch
    tmp = BIND + ".tmp.%d" % os.getpid()
    # libdfv.so is found beside the extension; torch's libraries are loaded by then
    cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", tmp, bind_obj, "-L", HERE, "-l:libdfv.so", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(os.path.dirname(torch.__file__), "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("linking the binding failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, BIND)
    with open(_stamp(), "w") as f:
        f.write(_torch())
    return LIB


if __name__ == "__main__":
    v = "-v" in sys.argv
    print(build(force=True, verbose=v, extra=(["-Xptxas", "-v"] if v else [])))
