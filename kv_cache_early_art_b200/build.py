"""Build libart.so in-tree (nvcc, sm_100a, CUDA runtime linked statically) and
the _marshal module, the binding's argument marshalling (g++, against torch).

The library is written for the B200 only: one architecture, no PTX fallback.
"""
from __future__ import annotations

import os
import re
import subprocess
import sys
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libart.so")
# one translation unit per group of walk instantiations, so that they compile in parallel
SOURCES = [os.path.join(CSRC, f) for f in ("art_api.cu", "art_order.cu", "art_walk_f32.cu", "art_walk_bf16.cu",
                                           "art_walk_mma.cu", "art_walk_multi.cu", "art_no_alloc.cu", "art_append.cu",
                                           "art_split.cu", "art_evict.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in ("art_kernels.cuh", "art_ptx.cuh", "art_host.h", "art_walk.h", "art_walk_dl.cuh", "art_walk_gr.cuh",
                                                  "art_stream.cuh")] + [
    os.path.join(ROOT, "include", "art.h")]

MARSHAL_DEPS = [os.path.join(CSRC, "art_marshal.cpp"), os.path.join(ROOT, "include", "art.h")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-std=c++17", "-lineinfo",
    "-Xcompiler", "-fPIC",
    "-Xptxas", "-warn-spills",
]
LINK_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-cudart", "static"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in DEPS)


def marshal_path() -> str:
    """The _marshal module's file, named after the torch and the Python it is
    built against: another version of either has a file of its own and never
    loads this one."""
    import torch
    version = re.sub(r"[^0-9A-Za-z]+", "_", str(torch.__version__))
    return os.path.join(HERE, f"_marshal.torch_{version}{sysconfig.get_config_var('EXT_SUFFIX')}")


def build_marshal(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/art_marshal.cpp into marshal_path() if it is missing or stale."""
    lib = marshal_path()
    if not force and os.path.exists(lib) and all(os.path.getmtime(p) <= os.path.getmtime(lib) for p in MARSHAL_DEPS):
        return lib
    import torch
    at = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc())) or "/usr/local/cuda"
    tmp = lib + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{sysconfig.get_paths()['include']}", f"-isystem{at}/include", f"-isystem{cuda}/include", "-o", tmp,
           MARSHAL_DEPS[0], f"-L{at}/lib", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd, cwd=CSRC)
    os.replace(tmp, lib)
    return lib


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/ into libart.so next to this file if it is missing or
    stale, then the _marshal module.  Where that one cannot be built (no g++, no
    Python headers) a warning says so: only the cache operators need it."""
    if force or stale():
        _build_libart(verbose)
    try:
        build_marshal(force=force, verbose=verbose)
    except (ImportError, OSError, subprocess.CalledProcessError) as e:
        warnings.warn(f"the _marshal module is not built, so the cache operators are not available: {e}")
    return LIB


def _build_libart(verbose: bool) -> None:
    """Every translation unit to an object in parallel, then one link."""
    import tempfile
    from concurrent.futures import ThreadPoolExecutor
    tmpdir = tempfile.mkdtemp(prefix="art_build_")
    objs = [os.path.join(tmpdir, os.path.basename(src)[:-3] + ".o") for src in SOURCES]

    def compile_one(pair):
        src, obj = pair
        cmd = [nvcc(), *NVCC_FLAGS, "-c", "-o", obj, src]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        r = subprocess.run(cmd, cwd=CSRC, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
        return cmd, r

    jobs = max(1, min(len(SOURCES), os.cpu_count() or 1))
    with ThreadPoolExecutor(jobs) as ex:
        results = list(ex.map(compile_one, zip(SOURCES, objs)))
    for cmd, r in results:
        if r.stdout:
            sys.stderr.write(r.stdout)
        if r.returncode != 0:
            raise subprocess.CalledProcessError(r.returncode, cmd, r.stdout)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc(), *LINK_FLAGS, "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd, cwd=CSRC)
    os.replace(tmp, LIB)
    for obj in objs:
        os.remove(obj)
    os.rmdir(tmpdir)


if __name__ == "__main__":
    print(build_library(force="--force" in sys.argv, verbose=True))
    build_marshal()                  # (raises where the library's call only warned)
