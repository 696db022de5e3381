"""Build libtlq.so (sm_103a) in-tree with nvcc: one object per .cu, compiled in
parallel, then one shared-library link; beside it, with the C compiler, the
Python module that shortens the serving calls and its way to read torch's
tensors (the library does without them where they cannot be built).  No cmake,
no torch extension."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
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
# how that module reads torch's tensors, for one version of torch (named in TENSORS_OF)
TENSORS = os.path.join(BUILD, "_tlq_tensors" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
TENSORS_OF = TENSORS + ".torch"

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


def build_tensors(force: bool = False) -> bool:
    """TENSORS: csrc/tensors.cpp against the headers of the torch that is installed
    (which is not imported).  Without them, or where it does not compile, the C
    API module reads tensors through their attributes."""
    src = os.path.join(CSRC, "tensors.cpp")
    spec = importlib.util.find_spec("torch")
    root = os.path.dirname(spec.origin) if spec and spec.origin else ""
    if not os.path.exists(os.path.join(root, "include", "torch", "csrc", "autograd", "python_variable.h")):
        return False
    with open(os.path.join(root, "version.py")) as f:
        version = re.search(r"""__version__ = ['"]([^'"]*)""", f.read())
    if not version:
        return False
    version = version.group(1)
    deps = [src, os.path.join(CSRC, "tensors.h"), os.path.abspath(__file__)]
    if not force and _fresh(TENSORS, deps) and os.path.exists(TENSORS_OF) and open(TENSORS_OF).read() == version:
        return True
    tmp = TENSORS + ".tmp%d" % os.getpid()
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], cuda, CSRC]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-w", "-shared", "-fPIC"] + ["-I" + i for i in include] + \
        [src, "-o", tmp, "-L" + os.path.join(root, "lib"), "-lc10", "-ltorch_cpu"]
    try:
        done = subprocess.run(cmd, capture_output=True, text=True).returncode == 0
    except OSError:
        done = False
    if not done:
        for path in (TENSORS, TENSORS_OF):  # of an older source or another torch
            if os.path.exists(path):
                os.remove(path)
        return False
    # the version only ever stands beside the library it is of: it goes first and comes back last, whole
    if os.path.exists(TENSORS_OF):
        os.remove(TENSORS_OF)
    os.replace(tmp, TENSORS)
    tmp = TENSORS_OF + ".tmp%d" % os.getpid()
    with open(tmp, "w") as f:
        f.write(version)
    os.replace(tmp, TENSORS_OF)
    return True


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every kernel source for sm_103a and link libtlq.so; return its path."""
    os.makedirs(BUILD, exist_ok=True)
    build_binding(force)
    if not force and up_to_date():
        build_tensors()
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

    with cf.ThreadPoolExecutor(max_workers=min(9, len(srcs) + 1)) as ex:
        tensors = ex.submit(build_tensors, force)
        results = list(ex.map(compile_one, srcs))
        tensors.result()
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
