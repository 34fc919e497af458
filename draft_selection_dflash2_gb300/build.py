"""Builds libdflash2.so (the CUDA kernels behind the C ABI) for sm_103a, in-tree,
and _dflash2_bind.so (the compiled half of the Python binding).

Each .cu file is compiled separately (in parallel) with nvcc and the objects
are linked into one shared library next to this file; the binding is one g++
call beside them.  Rebuilds only when a source or header is newer than the
library.
"""
import concurrent.futures
import glob
import os
import subprocess
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdflash2.so")
BIND = os.path.join(HERE, "_dflash2_bind.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")

NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) +
                  glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build_bind(force: bool = False) -> str:
    """The extension module that checks the cache operators' tensors and calls the C ABI (needs g++ and the headers of
    torch and Python)."""
    import sysconfig

    import torch
    torch_dir = os.path.dirname(torch.__file__)
    os.makedirs(BUILD, exist_ok=True)
    stamp = f"// torch {torch.__version__}, Python {sysconfig.get_python_version()}\n"
    stamp_file = os.path.join(BUILD, "bind.stamp")
    same = os.path.exists(stamp_file) and open(stamp_file).read() == stamp
    if not force and same and not _stale(BIND, [BIND_SRC, os.path.join(INCLUDE, "dflash2.h"), __file__]):
        return BIND
    include = os.path.join(torch_dir, "include")
    tmp = BIND + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f'-DDFLASH2_TORCH="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE, "-isystem", include,
           "-isystem", os.path.join(include, "torch", "csrc", "api", "include"), "-isystem",
           sysconfig.get_paths()["include"], BIND_SRC, "-o", tmp, "-L", os.path.join(torch_dir, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BIND_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BIND)
    with open(stamp_file, "w") as f:
        f.write(stamp)
    return BIND


def _try_bind(force: bool = False):
    try:
        build_bind(force)
    except (RuntimeError, OSError, ImportError) as e:
        warnings.warn(f"the cache operators' binding was not built, everything else was: {e}")


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Builds the library, which has to succeed, and the binding, without which only the cache operators are missing."""
    srcs, hdrs = _sources(), _headers()
    os.makedirs(BUILD, exist_ok=True)
    if not force and not _stale(LIB, srcs + hdrs + [__file__]):
        _try_bind()
        return LIB

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        if force or _stale(obj, [src] + hdrs + [__file__]):
            cmd = [NVCC, *ARCH, *FLAGS, *extra_flags, "-c", src, "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
            if verbose and (r.stdout or r.stderr):
                print(r.stdout + r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(srcs) + 1)) as ex:
        bind = ex.submit(_try_bind, force)
        objs = list(ex.map(compile_one, srcs))
        bind.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-ldl", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
