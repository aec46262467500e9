"""Builds the CUDA library in-tree: kernelized_causal_attention_gb300/_lib/liblinattn.so, and
beside it _front.so, the compiled calls from torch tensors to it.

Every translation unit is compiled for sm_103a only (GB300), in parallel, then
linked into one shared library with the static CUDA runtime; _front.so is host
code against the headers of Python and torch.  Run directly
(python -m kernelized_causal_attention_gb300._build) or through
__graft_entry__.build().
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIBDIR = os.path.join(HERE, "_lib")
LIB = os.path.join(LIBDIR, "liblinattn.so")
FRONT = os.path.join(LIBDIR, "_front.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) \
        + [os.path.join(CSRC, "front.cpp"), os.path.join(os.path.dirname(HERE), "include", "linattn.h"), __file__]


MANIFEST = os.path.join(LIBDIR, "sources.txt")


def _manifest() -> str:
    import torch
    return "\n".join([*(os.path.basename(f) for f in sources()), f"torch {torch.__version__}"])


def up_to_date() -> bool:
    """Both libraries exist, were built from the current set of sources (an
    added or removed file, or another torch, forces a rebuild) and are newer
    than every input."""
    if not all(os.path.exists(f) for f in (LIB, FRONT, MANIFEST)):
        return False
    with open(MANIFEST) as f:
        if f.read() != _manifest():
            return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(FRONT))
    return all(os.path.getmtime(d) <= t for d in _deps())


def _front_obj(cuda_home: str) -> str:
    import torch
    root = os.path.join(os.path.dirname(torch.__file__), "include")
    obj = os.path.join(LIBDIR, "front.o")
    dirs = [INCLUDE, root, os.path.join(root, "torch", "csrc", "api", "include"), sysconfig.get_paths()["include"],
            os.path.join(cuda_home, "include")]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{d}" for d in dirs), "-c",
          os.path.join(CSRC, "front.cpp"), "-o", obj], "front.cpp")
    return obj


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed on {what}:\n{r.stderr}")
    return r.stderr


def _link_front(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = FRONT + f".tmp{os.getpid()}"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{LIBDIR}", "-l:liblinattn.so", "-Wl,-rpath,$ORIGIN",
          f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"], "_front.so")
    os.replace(tmp, FRONT)


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    if not force and up_to_date():
        return LIB
    os.makedirs(LIBDIR, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(LIBDIR, os.path.basename(src)[:-3] + ".o")
        err = _run([cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj], src)
        if verbose and err:
            sys.stderr.write(err)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(len(sources()) + 1, os.cpu_count() or 1))) as ex:
        front = ex.submit(_front_obj, os.path.dirname(os.path.dirname(os.path.realpath(cc))))
        objs = list(ex.map(compile_one, sources()))
        front = front.result()
    tmp = LIB + f".tmp{os.getpid()}"
    _run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], "the library")
    os.replace(tmp, LIB)
    _link_front(front)
    with open(MANIFEST, "w") as f:
        f.write(_manifest())
    return LIB


if __name__ == "__main__":
    import time
    t0 = time.time()
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv,
                extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
    print(f"built in {time.time() - t0:.1f}s")
