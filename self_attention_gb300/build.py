"""Builds the sm_103a shared library libattn_gb300.so in-tree with nvcc.

Each .cu file is compiled as its own translation unit, in parallel, then linked into one
shared library under self_attention_gb300/_build/.  The CUDA runtime is linked statically, so that the
library loads wherever the driver is, without a toolkit (the shared one, PyTorch's own in a process that
has loaded it, was measured: the calls of csrc/binding.cpp take the same time with either).  The driver is
reached through cudaGetDriverEntryPointByVersion, so no -lcuda is needed.  The tensor-level calls of the
linear layers and the norm go through a small CPython extension beside the library (csrc/binding.cpp, g++).
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libattn_gb300.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
BINDING_PATH = os.path.join(BUILD_DIR, "attn_binding.so")   # CPython extension over the library and PyTorch

SOURCES = ["attn_api.cu", "attn_fwd.cu", "attn_bwd.cu", "vector_add.cu", "proj.cu", "unfused.cu", "linear.cu", "norm.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required to build libattn_gb300")
    return cand


BINDING_SOURCE = "binding.cpp"


def _newer(path: str, inputs) -> bool:
    """Whether `path` is there and newer than its inputs and this file."""
    inputs = [*inputs, os.path.join(INCLUDE, "attn.h"), os.path.abspath(__file__)]
    return os.path.exists(path) and os.path.getmtime(path) >= max(os.path.getmtime(f) for f in inputs)


def _library_fresh() -> bool:
    return _newer(LIB_PATH, [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != BINDING_SOURCE])


def _torch_dir() -> str:
    return importlib.util.find_spec("torch").submodule_search_locations[0]


def _binding_for() -> str:
    """What the binding is built against: this interpreter, and the PyTorch it imports."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sysconfig.get_config_var('SOABI')}\n{_torch_dir()}\n{f.read()}"


def _binding_fresh() -> bool:
    try:
        with open(BINDING_PATH + ".for") as f:
            same = f.read() == _binding_for()
    except OSError:
        return False
    return same and _newer(BINDING_PATH, [os.path.join(CSRC, BINDING_SOURCE)])


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _compile_binding(tool: str, tag: str) -> str:
    obj = os.path.join(BUILD_DIR, f"binding.{tag}.o")
    torch_inc = os.path.join(_torch_dir(), "include")
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(tool))), "include")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-I{INCLUDE}", f"-I{torch_inc}",
          f"-I{os.path.join(torch_inc, 'torch', 'csrc', 'api', 'include')}", f"-I{cuda_inc}",
          f"-I{sysconfig.get_paths()['include']}", "-c", os.path.join(CSRC, BINDING_SOURCE), "-o", obj],
         "g++ on binding.cpp")
    return obj


def _link_binding(obj: str, tag: str):
    lib = os.path.join(_torch_dir(), "lib")
    tmp = BINDING_PATH + f".{tag}.tmp"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{BUILD_DIR}", "-l:" + LIB_NAME, f"-L{lib}", "-ltorch_python", "-ltorch",
          "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"],
         "linking the binding")
    os.remove(obj)
    os.replace(tmp, BINDING_PATH)
    with open(BINDING_PATH + ".for", "w") as f:
        f.write(_binding_for())


def build_library(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) libattn_gb300.so alone, which takes nvcc and nothing of Python's or PyTorch's;
    returns its path."""
    if not force and _library_fresh():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    tool = nvcc()
    tag = f"{os.getpid()}"

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", f".{tag}.o"))
        cmd = [tool, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.append("-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    objs = [o for o, _ in results]
    tmp = LIB_PATH + f".{tag}.tmp"
    r = subprocess.run([tool, *ARCH, "-shared", "-o", tmp, *objs, "-ldl"], capture_output=True, text=True)
    for o in objs:
        os.remove(o)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    if verbose:
        for _, log in results:
            print(log)
    return LIB_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) the library and the Python binding; returns the path of libattn_gb300.so.  A
    binding that does not compile is an error, raised when the library is in its place."""
    if not force and _library_fresh() and _binding_fresh():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    tag = f"{os.getpid()}"
    with cf.ThreadPoolExecutor(1) as ex:    # beside the library's sources
        obj = ex.submit(_compile_binding, nvcc(), tag) if force or not _binding_fresh() else None
        build_library(force, verbose)
    if obj is not None:
        _link_binding(obj.result(), tag)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
