"""Build the CUDA library (libpkv.so) and its compiled binding in-tree for sm_103a.

Each translation unit under ``csrc/`` is compiled by nvcc in parallel and the
objects are linked into ``_build/libpkv.so`` (CUDA runtime linked statically,
the driver reached at run time, so the library also loads on a machine
without a GPU).  ``csrc/torch_binding.cpp`` is compiled by the host compiler
next to them and linked into ``_build/_pkv_torch.so``, an extension module that
calls the library.  Each of the two is rebuilt when one of its own sources or
headers is newer; the library needs neither torch nor Python headers, and is
built without the binding where they are missing.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(BUILD_DIR, "libpkv.so")
EXT_SOURCE = os.path.join(CSRC, "torch_binding.cpp")
EXT_PATH = os.path.join(BUILD_DIR, "_pkv_torch.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers() -> list[str]:
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def _newer(path: str, inputs: list[str]) -> bool:
    """Whether `path` exists and is no older than any of the inputs."""
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(p) <= t for p in inputs)


def library_up_to_date() -> bool:
    return _newer(LIB_PATH, sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _headers())


def binding_up_to_date() -> bool:
    return _newer(EXT_PATH, [EXT_SOURCE] + _headers())


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _run(cmd: list[str], what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what}:\n{r.stdout}\n{r.stderr}")
    return r.stdout + r.stderr


def build_library(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """libpkv.so alone: needs nvcc, neither torch nor Python headers."""
    if not force and library_up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    srcs = sources()
    objs = [os.path.join(BUILD_DIR, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(args):
        src, obj = args
        said = _run([nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj], f"nvcc failed on {os.path.basename(src)}")
        if verbose and said:
            print(said)

    with cf.ThreadPoolExecutor(max_workers=jobs or min(8, len(srcs))) as ex:
        list(ex.map(compile_one, zip(srcs, objs)))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], "nvcc link failed")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def _binding_flags() -> tuple[list[str], list[str]] | None:
    """The binding's compiler and linker flags; None where torch or its or Python's headers are missing."""
    try:
        import torch
    except ImportError:
        return None
    root = os.path.dirname(torch.__file__)
    inc, python = os.path.join(root, "include"), sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(python, "Python.h")) or not os.path.exists(os.path.join(inc, "ATen")):
        return None
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    return (["-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
             "-I", INCLUDE, "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"), "-I", cuda,
             "-I", python],
            ["-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"])


def build(force: bool = False, verbose: bool = False, jobs: int | None = None) -> str:
    """The library and, where torch's and Python's headers are installed, the compiled binding, each
    if it is out of date.  The library is in place whatever becomes of the binding."""
    flags = _binding_flags() if force or not binding_up_to_date() else None
    missing = flags is None and not binding_up_to_date()
    cxx, obj = os.environ.get("CXX", "g++"), os.path.join(BUILD_DIR, "torch_binding.o")
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:  # next to the library's sources
        compiled = flags and ex.submit(_run, [cxx, *flags[0], "-c", EXT_SOURCE, "-o", obj],
                                       f"{cxx} failed on {os.path.basename(EXT_SOURCE)}")
        build_library(force, verbose, jobs)
        if compiled:
            compiled.result()
    if flags:
        tmp = EXT_PATH + f".tmp{os.getpid()}"
        _run([cxx, "-shared", "-o", tmp, obj, *flags[1], "-L", BUILD_DIR, "-l:libpkv.so", "-Wl,-rpath,$ORIGIN"],
             "linking the binding failed")
        os.replace(tmp, EXT_PATH)
    elif missing:
        if os.path.exists(EXT_PATH):
            os.remove(EXT_PATH)  # of other sources than the library
        warnings.warn("torch's or Python's headers are missing: the compiled binding is not built, and the calls "
                      "that go through it will raise")
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
