"""Build step for the CUDA library: nvcc for sm_103a, in-tree.

``build()`` compiles ``csrc/*.cu`` (one translation unit each, in parallel) and
links ``_lib/libmoe_route.so``, and with g++ the Python calls of the decode-step
operators (``csrc/decode_ext.cpp``, against PyTorch's headers) into an extension
module beside it, with a note of the PyTorch that it was built against.  The
objects go to ``_build/``.
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_DIR = os.path.join(PKG, "_lib")
LIB_PATH = os.path.join(LIB_DIR, "libmoe_route.so")
EXT_SRC = os.path.join(CSRC, "decode_ext.cpp")
EXT_PATH = os.path.join(LIB_DIR, "moe_decode_ext" + sysconfig.get_config_var("EXT_SUFFIX"))
EXT_STAMP = EXT_PATH + ".torch"  # the PyTorch that it was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cuda_home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    cand = os.path.join(cuda_home, "bin", "nvcc")
    return cand if os.path.exists(cand) else (shutil.which("nvcc") or "nvcc")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [
        os.path.join(INCLUDE, "moe_route.h")]


def up_to_date() -> bool:
    """Whether the library is newer than its sources."""
    if not os.path.exists(LIB_PATH):
        return False
    t = os.path.getmtime(LIB_PATH)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _torch_abi() -> str:
    """What an extension module has to have been built against: this PyTorch."""
    import torch

    return f"torch {torch.__version__} cxx11 {int(torch._C._GLIBCXX_USE_CXX11_ABI)}\n"


def ext_abi_matches() -> bool:
    """Whether the extension module was built against the PyTorch that runs."""
    try:
        with open(EXT_STAMP) as f:
            return f.read() == _torch_abi()
    except OSError:
        return False


def ext_up_to_date() -> bool:
    """Whether the extension module is newer than its sources and fits this PyTorch."""
    if not os.path.exists(EXT_PATH) or not ext_abi_matches():
        return False
    t = os.path.getmtime(EXT_PATH)
    return all(os.path.getmtime(p) <= t for p in (EXT_SRC, os.path.join(INCLUDE, "moe_route.h")))


def _torch_flags():
    """Include, define and link flags for PyTorch's headers and libraries."""
    import torch

    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    return ["-I", sysconfig.get_paths()["include"], "-I", os.path.join(root, "include"),
            "-I", os.path.join(cuda, "include"),
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"], [
                "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python",
                f"-Wl,-rpath,{lib}"]


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stderr}")
    return r.stderr


def _link(cmd, path):
    """Run a link command (its output path left out) and put the result in place at once."""
    fd, tmp = tempfile.mkstemp(suffix=".so", dir=LIB_DIR)
    os.close(fd)
    try:
        _run([*cmd, "-o", tmp], "link failed")
    except BaseException:
        os.unlink(tmp)
        raise
    os.replace(tmp, path)


def _compile_ext() -> str:
    obj = os.path.join(BUILD_DIR, "decode_ext.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", *_torch_flags()[0], "-c", EXT_SRC, "-o", obj],
         f"g++ failed for {EXT_SRC}")
    return obj


def _build_lib(verbose) -> None:
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        return obj, _run(cmd, f"nvcc failed for {src}")

    with ThreadPoolExecutor(max_workers=8) as ex:
        results = list(ex.map(compile_one, _sources()))
    _link([nvcc, *ARCH, "-shared", "-cudart", "shared", *(o for o, _ in results),
           "-Xlinker", "-rpath=/usr/local/cuda/lib64"], LIB_PATH)
    if verbose:
        for _, log in results:
            print(log)


def build(force: bool = False, verbose: bool = False, extension: bool = True) -> str:
    """Compile what is older than its sources; return the library's path.

    The library comes first and needs nvcc only.  ``extension``: also the module
    of the decode-step calls, which needs g++ and PyTorch's C++ headers; without
    it everything but those calls runs."""
    lib = force or not up_to_date()
    ext = extension and (force or not ext_up_to_date())
    if not lib and not ext:
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    os.makedirs(LIB_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=1) as pool:
        ext_obj = pool.submit(_compile_ext) if ext else None
        if lib:
            _build_lib(verbose)
        if ext:
            obj = ext_obj.result()  # an error in it leaves the library built
            if os.path.exists(EXT_STAMP):
                os.unlink(EXT_STAMP)
            _link(["g++", "-shared", obj, "-L", LIB_DIR, "-lmoe_route", "-Wl,-rpath,$ORIGIN",
                   *_torch_flags()[1]], EXT_PATH)
            with open(EXT_STAMP, "w") as f:
                f.write(_torch_abi())
    return LIB_PATH
