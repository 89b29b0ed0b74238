"""Builds libkda_gb300.so in-tree with nvcc for sm_103a (one -gencode), and the CPython
module _marshal (g++, against the headers of the installed PyTorch)."""
from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "libkda_gb300.so"
LIB_PATH = os.path.join(PKG, LIB_NAME)
MARSHAL_SRC = os.path.join(PKG, "marshal.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "-Xptxas", "-warn-spills", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the KDA library needs the CUDA toolkit to build")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (sources() + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(INCLUDE, "*.h")) + [MARSHAL_SRC, os.path.abspath(__file__)])


def marshal_path() -> str:
    """The _marshal module's file.  It uses interfaces of the interpreter and of PyTorch that
    change between versions, so its name says which it was compiled for."""
    import torch
    return os.path.join(PKG, f"_marshal.{sys.implementation.cache_tag}-torch-{torch.__version__}.so")


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not os.path.exists(marshal_path()):
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(marshal_path()))
    return all(os.path.getmtime(p) <= t for p in _deps())


def marshal_command(out: str):
    """g++ command of the _marshal module."""
    torch_dir = importlib.util.find_spec("torch").submodule_search_locations[0]
    inc = [os.path.join(torch_dir, "include"),
           os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include"),
           sysconfig.get_paths()["include"]]
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-I", INCLUDE,
            *[x for p in inc for x in ("-isystem", p)], MARSHAL_SRC, "-o", out,
            "-L" + os.path.join(torch_dir, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile every csrc/*.cu in parallel and link the shared library."""
    if not force and up_to_date():
        return LIB_PATH
    # objects in a directory of this process's own, the library replaced
    # atomically: concurrent builders (one per rank) never clobber each other
    obj_dir = os.path.join(BUILD_DIR, f"p{os.getpid()}")
    os.makedirs(obj_dir, exist_ok=True)
    cc = nvcc()
    inc = ["-I", INCLUDE, "-I", CSRC]

    def compile_marshal(_):
        tmp = marshal_path() + f".tmp{os.getpid()}"
        r = subprocess.run(marshal_command(tmp), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed on marshal.cpp:\n{r.stdout}{r.stderr}")
        os.replace(tmp, marshal_path())

    def compile_one(src):
        obj = os.path.join(obj_dir, os.path.basename(src) + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, *inc, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    srcs = sources()
    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        marshal = ex.submit(compile_marshal, None)
        objs = list(ex.map(compile_one, srcs))
        marshal.result()
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}{r.stderr}")
    os.replace(tmp, LIB_PATH)
    shutil.rmtree(obj_dir, ignore_errors=True)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True))
