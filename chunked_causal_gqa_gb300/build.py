"""Build libpfa.so (the C-ABI library) for sm_103a with nvcc, and _pfa_torch.so
(the operators of the 8-bit and 4-bit caches on torch tensors, over that library) with g++, in-tree.

Each .cu under csrc/ is compiled to an object in parallel, then linked into
chunked_causal_gqa_gb300/_build/libpfa.so with the CUDA runtime linked
statically, so the library loads (and its symbols can be inspected) on a
machine without a GPU driver.
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import glob
import hashlib
import os
import shutil
import subprocess
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libpfa.so")
EXT = os.path.join(BUILD, "_pfa_torch.so")
EXT_KEY = os.path.join(BUILD, "_pfa_torch.key")
EXT_SOURCE = os.path.join(CSRC, "pfa_torch.cpp")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                     "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
                     "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpfa")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(INCLUDE, "pfa.h"), __file__]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def extension_environment() -> str:
    """The Python and torch that _pfa_torch.so is compiled against, in one line."""
    import sysconfig

    import torch
    return (f"{sysconfig.get_config_var('SOABI')} torch {torch.__version__} "
            f"{torch.version.git_version} cxx11abi {int(torch.compiled_with_cxx11_abi())}")


def _extension_key() -> str:
    """What _pfa_torch.so depends on: its environment, then its sources and this file."""
    h = hashlib.sha256()
    for path in (EXT_SOURCE, os.path.join(INCLUDE, "pfa.h"), __file__):
        with open(path, "rb") as f:
            h.update(f.read())
    return f"{extension_environment()}\n{h.hexdigest()}\n"


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def built_environment() -> str:
    """The environment that the present _pfa_torch.so was compiled against ("": unknown)."""
    return _read(EXT_KEY).partition("\n")[0]


def build_extension(force: bool = False) -> str:
    """Compile _pfa_torch.so against this Python's torch, unless it is up to date; returns its path.

    Raises RuntimeError or OSError where it cannot be compiled, and then leaves none."""
    import sysconfig

    import torch
    key = _extension_key()
    if not force and os.path.exists(EXT) and _read(EXT_KEY) == key:
        return EXT
    for stale in (EXT_KEY, EXT):
        with contextlib.suppress(FileNotFoundError):
            os.remove(stale)
    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    dirs = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api",
                                                        "include"),
            os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = EXT + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", EXT_SOURCE, "-o", tmp]
    for d in dirs:
        cmd += ["-isystem", d]
    cmd += ["-L", BUILD, "-L", os.path.join(base, "lib"), "-lpfa", "-ltorch_python", "-ltorch_cpu",
            "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {EXT_SOURCE}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, EXT)
    with open(tmp, "w") as f:
        f.write(key)
    os.replace(tmp, EXT_KEY)
    return EXT


def _extension_or_warning(force: bool) -> None:
    """libpfa.so serves C callers and the 16/32-bit path without the extension."""
    try:
        build_extension(force)
    except (OSError, RuntimeError) as e:
        warnings.warn("_pfa_torch.so was not built, so the Python functions of the 8-bit cache's "
                      f"operators will raise ImportError: {e}", stacklevel=3)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link libpfa.so, then _pfa_torch.so; returns libpfa.so's path.

    Where _pfa_torch.so cannot be compiled (no g++, no headers of Python or torch) that is a
    warning: only the operators of the 8-bit and 4-bit caches need it, and only from Python."""
    if not force and not extra_flags and up_to_date():
        _extension_or_warning(force)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc] + NVCC_FLAGS + list(extra_flags) + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(compile_one, _sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-Xlinker",
                         "-soname=libpfa.so", "-o", tmp] + objs + \
        ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _extension_or_warning(force)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force=True, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "-v" in sys.argv else []))
