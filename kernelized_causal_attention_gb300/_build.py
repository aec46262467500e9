"""Builds the CUDA library in-tree: kernelized_causal_attention_gb300/_lib/liblinattn.so, and
beside it _front.so, the compiled calls from torch tensors to it.

Every translation unit is compiled for sm_103a only (GB300), in parallel, then
linked into one shared library with the static CUDA runtime: library(), which needs
nvcc and its host compiler only.  _front.so is host code against the headers of
Python and torch, and linked to that library; where it cannot be built, build() says
so with the library in place.  Run directly
(python -m kernelized_causal_attention_gb300._build, with --library for the library
alone) or through __graft_entry__.build().
"""
from __future__ import annotations

import contextlib
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
        + [os.path.join(INCLUDE, "linattn.h"), __file__]


def _front_deps():
    return [os.path.join(CSRC, "front.cpp"), os.path.join(INCLUDE, "linattn.h"), __file__]


MANIFEST = os.path.join(LIBDIR, "sources.txt")
FRONT_MANIFEST = os.path.join(LIBDIR, "front.txt")


def _manifest() -> str:
    return "\n".join(os.path.basename(f) for f in sources())


def front_manifest() -> str:
    """What _front.so is good for: the torch and the Python whose headers it was compiled against."""
    import torch
    return f"torch {torch.__version__}\npython {sys.version_info.major}.{sys.version_info.minor}"


def _newest(lib, deps) -> bool:
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in deps)


def _current(lib, manifest, said, deps) -> bool:
    """lib exists, was built from what the manifest says and is newer than every input."""
    if not (os.path.exists(lib) and os.path.exists(manifest)):
        return False
    with open(manifest) as f:
        return f.read() == said and _newest(lib, deps)


def up_to_date() -> bool:
    """The library exists, was built from the current set of sources (an
    added or removed file forces a rebuild) and is newer than every input."""
    return _current(LIB, MANIFEST, _manifest(), _deps())


def front_up_to_date() -> bool:
    """The same of _front.so, which another torch or Python makes out of date."""
    return _current(FRONT, FRONT_MANIFEST, front_manifest(), _front_deps())


def _front_obj() -> str:
    import torch
    cuda_home = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
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


def _say(manifest, text) -> None:
    """Whole or not at all, for a process that reads it meanwhile."""
    tmp = manifest + f".tmp{os.getpid()}"
    with open(tmp, "w") as f:
        f.write(text)
    os.replace(tmp, manifest)


def _link_front(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = FRONT + f".tmp{os.getpid()}"
    _run([os.environ.get("CXX", "g++"), "-shared", "-o", tmp, obj, f"-L{LIBDIR}", "-l:liblinattn.so", "-Wl,-rpath,$ORIGIN",
          f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"], "_front.so")
    os.replace(tmp, FRONT)
    _say(FRONT_MANIFEST, front_manifest())


def _link(cc, objs) -> None:
    if os.path.exists(FRONT_MANIFEST) and not (os.path.exists(FRONT) and _newest(FRONT, _front_deps())):
        with contextlib.suppress(FileNotFoundError):  # another process that builds
            os.remove(FRONT_MANIFEST)  # a front of another header than the library's is not to be loaded
    tmp = LIB + f".tmp{os.getpid()}"
    _run([cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs], "the library")
    os.replace(tmp, LIB)
    _say(MANIFEST, _manifest())


def _build(ex, force, verbose, extra) -> None:
    """The library, its units compiled by the executor."""
    if not force and up_to_date():
        return
    os.makedirs(LIBDIR, exist_ok=True)
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(LIBDIR, os.path.basename(src)[:-3] + ".o")
        err = _run([cc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj], src)
        if verbose and err:
            sys.stderr.write(err)
        return obj

    _link(cc, list(ex.map(compile_one, sources())))


def _executor():
    return ThreadPoolExecutor(max_workers=max(1, min(len(sources()) + 1, os.cpu_count() or 1)))


def library(force: bool = False, verbose: bool = False, extra=()) -> str:
    """The CUDA library alone."""
    with _executor() as ex:
        _build(ex, force, verbose, extra)
    return LIB


def build(force: bool = False, verbose: bool = False, extra=()) -> str:
    """The CUDA library, and _front.so beside it; the library's path."""
    if not force and up_to_date() and front_up_to_date():
        return LIB
    os.makedirs(LIBDIR, exist_ok=True)
    with _executor() as ex:
        # compiled beside the library's units, waited for (and refused) once the library is linked
        front = ex.submit(_front_obj) if force or not front_up_to_date() else None
        _build(ex, force, verbose, extra)
        if front is not None:
            try:
                _link_front(front.result())
            except Exception as e:
                raise RuntimeError(f"{LIB} is built; _front.so, which the calls from gated_fwd on go through, is not: {e}") from e
    return LIB


if __name__ == "__main__":
    import time
    t0 = time.time()
    print((library if "--library" in sys.argv else build)(force="--force" in sys.argv, verbose="-v" in sys.argv,
                                                          extra=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
    print(f"built in {time.time() - t0:.1f}s")
