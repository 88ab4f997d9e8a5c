"""Build libkvz.so (sm_100a) in-tree with nvcc.

    python -m query_agnostic_kv_kvz_b200.build [--force]

Compiles every ``csrc/*.cu`` with ``-gencode arch=compute_100a,code=sm_100a``
and links them into ``query_agnostic_kv_kvz_b200/libkvz.so``.  The CUDA
runtime is linked statically; the driver's tensor-map encoder is looked up at
run time, so the library needs no libcuda at link time.

``csrc/fast_calls.cpp`` becomes ``_kvz_fast`` (with the interpreter's suffix),
a CPython module for the installed torch that shortens the host's part of the
decoding calls.  The binding works without it, only slower, so a machine that
cannot compile it (no Python headers, say) is told and goes on, without the
module of an earlier build: it calls the C ABI of the header that it was
compiled with, which the binding compares with the one there is.
"""
from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libkvz.so")
OBJDIR = os.path.join(ROOT, "_build")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC,-O2",
    "-I" + INCLUDE, "-I" + CSRC,
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; the KVzip CUDA library cannot be built")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(p) <= t for p in _deps())


FAST_SRC = os.path.join(CSRC, "fast_calls.cpp")
FAST = os.path.join(PKG, "_kvz_fast" + sysconfig.get_config_var("EXT_SUFFIX"))
FAST_STAMP = os.path.join(OBJDIR, "fast_calls.torch")


def header_id() -> str:
    """A name for the C ABI: the hash of the header that declares it."""
    with open(os.path.join(INCLUDE, "kvz.h"), "rb") as f:
        return hashlib.sha256(f.read()).hexdigest()[:32]


def build_fast(force: bool = False, verbose: bool = False) -> bool:
    """Compile (if stale) the host module; False where it cannot be compiled."""
    import torch
    stamp = "%s %s" % (torch.__version__, sys.version)
    if not force and os.path.exists(FAST) and os.path.exists(FAST_STAMP) and open(FAST_STAMP).read() == stamp and \
            all(os.path.getmtime(p) <= os.path.getmtime(FAST) for p in (FAST_SRC, os.path.join(INCLUDE, "kvz.h"))):
        return True
    t = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = FAST + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI),
           "-DKVZ_TORCH_VERSION=\"%s\"" % torch.__version__, "-DKVZ_HEADER_ID=\"%s\"" % header_id(),
           "-I" + os.path.join(t, "include"), "-I" + os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include"), "-I" + INCLUDE, FAST_SRC,
           "-o", tmp, "-L" + os.path.join(t, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10",
           "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd))
    # nothing of an earlier build is left to be imported should this one fail
    for old in glob.glob(os.path.join(os.path.dirname(FAST), "_kvz_fast*.so")) + [FAST_STAMP]:
        if os.path.exists(old):
            os.remove(old)
    try:
        subprocess.run(cmd, check=True)
    except (OSError, subprocess.CalledProcessError) as e:
        print("kvz: %s not built (%s); the decoding calls take their slower way on the host" % (FAST, e),
              file=sys.stderr)
        return False
    os.replace(tmp, FAST)
    os.makedirs(OBJDIR, exist_ok=True)
    with open(FAST_STAMP, "w") as f:
        f.write(stamp)
    return True


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and return the path of libkvz.so."""
    build_library(force, verbose)
    build_fast(force, verbose)                        # behind the library whose calls it makes
    return LIB


def build_library(force: bool = False, verbose: bool = False) -> None:
    if not force and up_to_date():
        return
    nvcc = _nvcc()
    os.makedirs(OBJDIR, exist_ok=True)
    objs = []
    for src in _sources():
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        subprocess.run(cmd, check=True)
        objs.append(obj)
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp, *objs,
           "-cudart", "static"]
    if verbose:
        print(" ".join(cmd))
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
