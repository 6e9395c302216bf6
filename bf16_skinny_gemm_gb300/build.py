"""Build the CUDA library ``libsgemm_skinny.so`` in-tree with nvcc for sm_103a.

Each translation unit is compiled in parallel (``nvcc -c``), then linked into
one shared library with the CUDA runtime linked statically, so the library
needs nothing but the NVIDIA driver at run time.  Output goes to
``bf16_skinny_gemm_gb300/_build/``.

Beside it, the host compiler builds ``_marshal.*.so`` (``native/marshal.cpp``), the short way from
torch tensors to the decode operators' calls, against the installed torch; its name says which.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libsgemm_skinny.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
MARSHAL_SRC = os.path.join(PKG, "native", "marshal.cpp")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
COMMON_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
                "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _deps() -> list[str]:
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(CSRC, "*.inc")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def is_stale() -> bool:
    return _stale(LIB_PATH, _deps())


def marshal_path() -> str:
    """Where the module for this Python and torch is.  It reads tensors by torch's own layout of
    them, so one built against another torch is another file."""
    import torch

    build = f"{torch.version.git_version} {torch._C._GLIBCXX_USE_CXX11_ABI}"
    return os.path.join(BUILD_DIR, f"_marshal.{sysconfig.get_config_var('SOABI')}.torch-{torch.__version__}-"
                                   f"{hashlib.sha1(build.encode()).hexdigest()[:8]}.so")


def build_marshal(force: bool = False) -> str:
    """Compile ``native/marshal.cpp`` if it, Python or torch changed; returns the module's path."""
    path = marshal_path()
    deps = [MARSHAL_SRC, *glob.glob(os.path.join(INCLUDE, "*.h"))]
    if not force and not _stale(path, deps):
        return path
    import torch

    os.makedirs(BUILD_DIR, exist_ok=True)
    home = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    inc = [INCLUDE, os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], cuda]
    tmp = path + f".tmp{os.getpid()}"
    cmd = ["g++", "-std=c++17", "-O2", "-fPIC", "-shared", *[f for d in inc for f in ("-isystem", d)], MARSHAL_SRC,
           "-o", tmp, "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {MARSHAL_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link the library if any source changed; returns its path."""
    if not force and not is_stale():
        build_marshal()
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH_FLAGS, *COMMON_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stdout + r.stderr

    srcs = sources()
    workers = max(1, min(len(srcs), os.cpu_count() or 4))
    with cf.ThreadPoolExecutor(workers) as ex:
        marshal = ex.submit(build_marshal, force)
        results = list(ex.map(compile_one, srcs))
        marshal.result()
    if verbose or ptxas_info:
        for _, log in results:
            if log.strip():
                print(log)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH_FLAGS, "-shared", "-cudart", "static", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
