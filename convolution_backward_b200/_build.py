"""Build libdgrad.so (and libdgrad_debug.so) in-tree with nvcc for sm_100a.

Every .cu file under csrc/ is compiled to an object in _build/ (in parallel),
then linked into convolution_backward_b200/libdgrad.so with the CUDA runtime
linked statically.  ptxas register/spill reports go to _build/ptxas.log.  The
same sources built with -DDGRAD_DEBUG (objects in _build/debug/) give
libdgrad_debug.so, whose kernels check every hand-indexed store against its
output buffer.  csrc/tensor_lists.cpp, the binding's reader of tensor lists, becomes the Python
extension module convolution_backward_b200/_tensor_lists (g++, torch's headers), and is left out where there is no
torch: the libraries need none.  Rebuilds only when a source, header or this file is newer than a library, and the
module also when torch or Python is another.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libdgrad.so")
LIB_DEBUG = os.path.join(PKG, "libdgrad_debug.so")

LISTS = os.path.join(PKG, "_tensor_lists" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))   # this Python's
LISTS_FOR = os.path.join(BUILD, "tensor_lists.torch")      # the torch that it was built against
LISTS_SRC = os.path.join(CSRC, "tensor_lists.cpp")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
                 "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = srcs + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return srcs, deps


def needs_build() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(LIB_DEBUG):
        return True
    _, deps = _inputs()
    t = min(os.path.getmtime(LIB), os.path.getmtime(LIB_DEBUG))
    return any(os.path.getmtime(d) > t for d in deps)


def _torch():
    """(package folder, version) of the installed torch, or None."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "unknown"
    return list(spec.submodule_search_locations)[0], version


def lists_need_build() -> bool:
    if not os.path.exists(LISTS) or not os.path.exists(LISTS_FOR):
        return True
    with open(LISTS_FOR) as f:
        if f.read() != _torch()[1]:
            return True
    return any(os.path.getmtime(f) > os.path.getmtime(LISTS) for f in (LISTS_SRC, os.path.abspath(__file__)))


def _build_lists() -> None:
    root, version = _torch()
    tmp = LISTS + f".tmp{os.getpid()}"
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", *[f"-I{i}" for i in inc], LISTS_SRC, "-o", tmp,
           "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {LISTS_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LISTS)
    os.makedirs(BUILD, exist_ok=True)
    with open(LISTS_FOR, "w") as f:
        f.write(version)
    untagged = os.path.join(PKG, "_tensor_lists.so")       # one that any Python would load
    if untagged != LISTS and os.path.exists(untagged):
        os.remove(untagged)


def build(force: bool = False, verbose: bool = False) -> str:
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        lists = None
        if _torch() is None:
            print("no torch: the Python binding's _tensor_lists module is not built")
        elif force or lists_need_build():
            lists = ex.submit(_build_lists)
        if force or needs_build():
            _build_kernels()
        if lists is not None:
            lists.result()
    if verbose:
        print(f"built {LIB}")
    return LIB


def _build_kernels() -> None:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    srcs, _ = _inputs()

    debug_dir = os.path.join(BUILD, "debug")
    os.makedirs(debug_dir, exist_ok=True)

    def compile_one(job):
        src, debug = job
        obj = os.path.join(debug_dir if debug else BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc, *CFLAGS, *(["-DDGRAD_DEBUG"] if debug else []), "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    jobs = [(s, False) for s in srcs] + [(s, True) for s in srcs]
    with cf.ThreadPoolExecutor(max_workers=min(16, os.cpu_count() or 4)) as ex:
        results = list(ex.map(compile_one, jobs))
    release, debug = results[:len(srcs)], results[len(srcs):]
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        for (obj, log), src in zip(release, srcs):
            f.write(f"==== {os.path.basename(src)}\n{log}\n")
    for lib, objs in ((LIB, release), (LIB_DEBUG, debug)):
        tmp = lib + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *[o for o, _ in objs],
               "-ldl", "-lpthread", "-lrt"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, lib)


if __name__ == "__main__":
    build(force=True, verbose=True)
