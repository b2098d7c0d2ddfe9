"""Build libgdn.so (the CUDA kernels behind the C ABI in include/gdn.h) for sm_100a.

    python -m gated_deltanet_mixer_verify_b200.build [--force]

Each csrc/*.cu file is compiled by nvcc (in parallel) and linked into the package
directory, next to this file, with the CUDA runtime linked statically so that the
library loads on machines without a GPU. _binding.so beside it (csrc/binding.cpp, by the host
compiler, against PyTorch's headers) is the native half of gdn.py's argument checks. It is built after
the library, and left out where PyTorch or Python's headers are missing: users of the C ABI need nvcc alone.
"""
import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdn.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_binding.so")
CXX = os.environ.get("CXX", "g++")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)])


def needs_build() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [NVCC] + ARCH + FLAGS + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def binding_versions() -> str:
    """What _binding.so is built against. It reads PyTorch's C++ objects, so it serves no other."""
    import torch
    return "PyTorch %s, %s, C++ ABI %d" % (torch.__version__, sysconfig.get_config_var("SOABI"), torch._C._GLIBCXX_USE_CXX11_ABI)


def binding_is_stale() -> bool:
    """Whether _binding.so is missing, older than its source, or built against other versions (the stamp beside it)."""
    try:
        with open(BINDING + ".for") as f:
            versions = f.read()
        built = os.path.getmtime(BINDING)
    except OSError:
        return True
    return versions != binding_versions() or built < max(os.path.getmtime(BINDING_SRC), os.path.getmtime(os.path.abspath(__file__)))


def build_binding(force: bool = False) -> str:
    """Compile _binding.so if it is stale; return its path."""
    if not force and not binding_is_stale():
        return BINDING
    import torch
    base = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp.%d" % os.getpid()
    cmd = [CXX, "-O2", "-std=c++17", "-shared", "-fPIC", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-DGDN_BUILT_FOR=\"%s\"" % binding_versions(), "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(base, "include"),
           "-I" + os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I" + os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), BINDING_SRC, "-o", tmp,
           "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed on %s:\n%s%s" % (CXX, BINDING_SRC, r.stdout, r.stderr))
    os.replace(tmp, BINDING)
    with open(BINDING + ".for", "w") as f:
        f.write(binding_versions())
    return BINDING


def binding_lacks() -> str:
    """What _binding.so needs and this machine does not have ("" if nothing)."""
    if importlib.util.find_spec("torch") is None:
        return "PyTorch"
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return "Python.h"
    return "" if shutil.which(CXX) else "a host compiler (%s)" % CXX


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libgdn.so (and _binding.so) if any source is newer than it; return its path."""
    lib = build_library(force, verbose)
    lacks = binding_lacks()
    if lacks:
        print("_binding.so not built, no %s: libgdn.so serves its C ABI; the Python binding needs both" % lacks, file=sys.stderr)
    else:
        build_binding(force)
    return lib


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libgdn.so, with nvcc alone; return its path."""
    if not force and not needs_build():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs), os.cpu_count() or 1))) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), srcs))
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [NVCC] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
