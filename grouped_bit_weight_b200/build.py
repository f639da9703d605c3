"""Builds libgbw.so (the sm_100a CUDA library) and _host.so (the Python module
of its short calls) in-tree.

Each .cu file compiles to its own object in parallel, then nvcc links the
shared library next to this file; g++ compiles the module against it and
torch.  No GPU is needed to build.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libgbw.so")
HOST_SRC = os.path.join(CSRC, "host.cpp")
HOST = os.path.join(HERE, "_host.so")
HOST_STAMP = os.path.join(BUILD, "host.txt")  # what _host.so was built against
HEADER = os.path.join(HERE, "..", "include", "gbw.h")

NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
         "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + [HEADER, __file__])


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose:
        sys.stderr.write(r.stderr)
    return obj


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in _deps())


def _host_stamp() -> str:
    import torch
    return f"torch {torch.__version__}, cuda {torch.version.cuda}, python {sys.version}"


def host_up_to_date() -> bool:
    """Whether _host.so is newer than its sources and of this torch and Python."""
    if not os.path.exists(HOST) or not os.path.exists(HOST_STAMP):
        return False
    t = os.path.getmtime(HOST)
    with open(HOST_STAMP) as f:
        return (f.read() == _host_stamp()
                and all(os.path.getmtime(d) <= t for d in (HOST_SRC, HEADER, __file__)))


def _host(force: bool) -> None:
    """_host.so: against torch's headers, linked to libgbw.so beside it."""
    if not force and host_up_to_date():
        return
    import torch
    os.makedirs(BUILD, exist_ok=True)
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(NVCC) or NVCC)))
    inc = [os.path.join(root, "include"), os.path.join(root, "include/torch/csrc/api/include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = HOST + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC",
           "-fvisibility=hidden", "-w", *(f"-I{d}" for d in inc),
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", HOST_SRC,
           "-o", tmp, f"-L{HERE}", "-l:libgbw.so", f"-L{os.path.join(root, 'lib')}", "-lc10",
           "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {HOST_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, HOST)
    with open(HOST_STAMP, "w") as f:
        f.write(_host_stamp())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        _host(force)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        objs = list(ex.map(lambda s: _compile(s, verbose), _sources()))
    tmp = LIB + ".tmp"
    cmd = [NVCC, *ARCH, "-shared", "-Xcompiler", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _host(force)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
