"""Build liblf_decode.so (sm_103a) in-tree with nvcc.

Each .cu file compiles to an object in parallel, then one shared library is
linked. Output: decode_kv_cache_step_gb300/lib/liblf_decode.so, and beside it
_lf_check.so, the binding's argument checks as an extension of the installed
torch (left out, with a warning, where it does not compile: the binding then
checks in Python). Nothing is installed outside the package directory.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
import tempfile
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "lib")
LIB_PATH = os.path.join(LIB_DIR, "liblf_decode.so")
CHECK_PATH = os.path.join(LIB_DIR, "_lf_check.so")
CHECK_SRC = os.path.join(CSRC, "lf_check.cpp")
OBJ_DIR = os.path.join(PKG, "_build")
STAMP_PATH = os.path.join(OBJ_DIR, "_lf_check.torch")  # the torch version CHECK_PATH is for

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC] + ARCH


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build liblf_decode.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps())


def check_up_to_date() -> bool:
    """Whether lib/_lf_check.so was compiled from the present source against the
    installed torch (the build notes its version)."""
    try:
        import torch
        with open(STAMP_PATH) as f:
            same = f.read() == torch.__version__
        t = os.path.getmtime(CHECK_PATH)
        return same and all(os.path.getmtime(p) <= t for p in (CHECK_SRC, __file__))
    except Exception:  # missing, or no usable torch: _build_check says so
        return False


def _build_check() -> None:
    """lib/_lf_check.so, against the installed torch; a warning where that fails."""
    tmp = None
    try:
        import torch

        base = os.path.dirname(torch.__file__)
        include = os.path.join(base, "include")
        for path in (LIB_DIR, OBJ_DIR):
            os.makedirs(path, exist_ok=True)
        for path in (STAMP_PATH, CHECK_PATH):
            if os.path.exists(path):
                os.unlink(path)
        fd, tmp = tempfile.mkstemp(suffix=".so", dir=LIB_DIR)
        os.close(fd)
        cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-w",
               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
               f'-DLF_TORCH_VERSION="{torch.__version__}"', "-I", include,
               "-I", os.path.join(include, "torch", "csrc", "api", "include"),
               "-I", sysconfig.get_paths()["include"], CHECK_SRC, "-o", tmp,
               "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(r.stderr[-400:])
        os.replace(tmp, CHECK_PATH)
        with open(STAMP_PATH, "w") as f:
            f.write(torch.__version__)
    except Exception as e:
        if tmp is not None and os.path.exists(tmp):
            os.unlink(tmp)
        warnings.warn(f"_lf_check.so was not built: {e}")


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile every kernel and the C ABI into liblf_decode.so; return its path. The
    argument checks beside it are compiled where they are missing or stale."""
    check_stale = force or not check_up_to_date()
    if not force and up_to_date():
        if check_stale:
            _build_check()
        return LIB_PATH
    os.makedirs(LIB_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        cmd = [cc, "-c", src, "-o", obj] + NVCC_FLAGS + extra
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stderr)
        return obj

    srcs = _sources()
    with ThreadPoolExecutor(max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        check = ex.submit(_build_check) if check_stale else None
        objs = list(ex.map(compile_one, srcs))
        if check is not None:
            check.result()
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=LIB_DIR)
    os.close(fd)
    cmd = [cc, "-shared", "-o", tmp] + objs + ARCH + ["-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        os.unlink(tmp)
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
