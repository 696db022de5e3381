"""Build libtlq.so (sm_103a) in-tree with nvcc: one object per .cu, compiled in
parallel, then one shared-library link; beside it, with the C compiler, the
Python module that shortens the serving calls (the library does without it
where it cannot be built).  No cmake, no torch extension."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libtlq.so")
# one file for each interpreter that uses the tree
BINDING = os.path.join(BUILD, "_tlq_binding" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-rdc=true", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-Wall", "-I" + INCLUDE]


def _nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + \
        sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)]


def _fresh(path, deps) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in deps)


def up_to_date() -> bool:
    return _fresh(LIB, _deps())


def build_binding(force: bool = False) -> bool:
    """BINDING: the C API module of the serving calls (host code only).  Without
    a C compiler or Python's headers there is none, and those calls go through
    ctypes."""
    src = os.path.join(CSRC, "binding.c")
    if not force and _fresh(BINDING, [src, os.path.join(INCLUDE, "tlq.h"), os.path.abspath(__file__)]):
        return True
    tmp = BINDING + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CC", "gcc"), "-O2", "-std=c11", "-Wall", "-shared", "-fPIC",
           "-I" + sysconfig.get_paths()["include"], src, "-o", tmp]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = r.stderr or "exit status %d" % r.returncode if r.returncode else ""
    except OSError as e:
        why = str(e)
    if why:
        if os.path.exists(BINDING):  # of an older source
            os.remove(BINDING)
        warnings.warn("no C API module, the serving calls will take longer: %s\n%s" % (" ".join(cmd), why))
        return False
    os.replace(tmp, BINDING)
    return True


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every kernel source for sm_103a and link libtlq.so; return its path."""
    os.makedirs(BUILD, exist_ok=True)
    build_binding(force)
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    srcs = _sources()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc] + NVCC_FLAGS + list(extra_flags) + ["-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr))
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(compile_one, srcs))
    if verbose:
        for _, log in results:
            print(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp%d" % os.getpid()
    cuda_lib = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "lib64") if os.path.isabs(nvcc) else ""
    rpath = ["-Xlinker", "-rpath=" + cuda_lib] if cuda_lib else []
    cmd = [nvcc] + ARCH + ["-shared", "-rdc=true", "-cudart", "shared", "-Xcompiler", "-fPIC"] + rpath + objs + \
        ["-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
