"""Builds libidx.so in-tree from csrc/*.cu with nvcc for sm_103a, and
_serving.so, the compiled part of the Python binding, from csrc/serving_py.cpp
with g++ against PyTorch's headers.

Each translation unit compiles in parallel; the objects go to _build/ and the
shared libraries next to this file.  A rebuild is skipped when the libraries are
newer than every source and header.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libidx.so")
EXT = os.path.join(HERE, "_serving.so")
EXT_SOURCE = os.path.join(CSRC, "serving_py.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
         "-Xcompiler", "-fvisibility=hidden",
         f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + [EXT_SOURCE] + glob.glob(os.path.join(CSRC, "*.cuh")) +
            glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")) +
            [os.path.abspath(__file__)])


def up_to_date() -> bool:
    if not (os.path.exists(LIB) and os.path.exists(EXT)):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr.strip():
            print(r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        ext = ex.submit(compile_serving, nvcc)
        objs = list(ex.map(compile_one, srcs))
    # libidx.so first: it does not depend on PyTorch, whatever becomes of the other
    tmp = LIB + f".tmp{os.getpid()}"
    _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], "link")
    os.replace(tmp, LIB)
    link_serving(*ext.result())
    return LIB


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def compile_serving(nvcc):
    """The binding's object file, and the folder of the PyTorch it was compiled against."""
    import torch
    torch_dir = os.path.dirname(torch.__file__)
    cuda_include = os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")
    obj = os.path.join(BUILD, "serving_py.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          f"-I{INCLUDE}", f"-isystem{torch_dir}/include",
          f"-isystem{torch_dir}/include/torch/csrc/api/include",
          f"-isystem{sysconfig.get_paths()['include']}", f"-isystem{cuda_include}",
          "-c", EXT_SOURCE, "-o", obj], f"g++ on {EXT_SOURCE}")
    return obj, torch_dir


def link_serving(obj, torch_dir):
    tmp = EXT + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{HERE}", "-l:libidx.so", f"-L{torch_dir}/lib",
          "-ltorch_python", "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
          "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{torch_dir}/lib"], "link of the serving binding")
    os.replace(tmp, EXT)


if __name__ == "__main__":
    print(build(force=True, verbose=True))
