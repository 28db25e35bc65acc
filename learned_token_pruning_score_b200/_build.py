"""Builds libtokengate.so in-tree with nvcc for sm_100a.

    python learned_token_pruning_score_b200/_build.py   (or __graft_entry__.build())

Each .cu under csrc/ is compiled to an object under _build/ (in parallel,
skipped when up to date), then linked into a shared library next to this
file. The CUDA runtime is linked statically, so the library loads on a
machine without a GPU driver (its exported symbols can be checked there).
csrc/binding.cpp becomes the extension module _binding, which the package
calls the library's per-token entry points through; it is built against the
torch that runs this.
"""

from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libtokengate.so")
BINDING = os.path.join(HERE, "_binding.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills", "-I", CSRC, "-I", INCLUDE]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put CUDA's bin on PATH)")


def _newer(src: str, dst: str, deps) -> bool:
    if not os.path.exists(dst):
        return True
    t = os.path.getmtime(dst)
    return any(os.path.getmtime(p) > t for p in [src, *deps])


def build(verbose: bool = False, force: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
                     + glob.glob(os.path.join(INCLUDE, "*.h")))
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        if force or _newer(src, obj, headers):
            cmd = [cc, *ARCH, *FLAGS, "-c", src, "-o", obj]
            if verbose:
                print(" ".join(cmd), flush=True)
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
            if verbose and (r.stderr.strip() or r.stdout.strip()):
                print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        objs = list(ex.map(compile_one, sources))
    if force or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB)
                                               for o in objs):
        cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", LIB, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    build_binding(verbose, force)
    return LIB


CXX_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared", "-DNDEBUG"]
BINDING_LIBS = ["-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def build_binding(verbose: bool = False, force: bool = False) -> str:
    """Builds _binding.so when its sources, or what its binary interface comes
    from (torch, Python, the compiler and its flags), are not those it was
    built from; the latter stand in a stamp beside the objects."""
    import sysconfig

    import torch

    src = os.path.join(CSRC, "binding.cpp")
    cxx = os.environ.get("CXX", "g++")
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    made_for = "\n".join([f"torch {torch.__version__}", f"python {sys.version}",
                          " ".join([cxx, *CXX_FLAGS, abi, *BINDING_LIBS])])
    stamp = os.path.join(BUILD, "binding.stamp")
    same = False
    if os.path.exists(stamp):
        with open(stamp) as f:
            same = f.read() == made_for
    if (same and not force
            and not _newer(src, BINDING, [LIB, os.path.join(INCLUDE, "tokengate.h")])):
        return BINDING
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    cmd = [cxx, *CXX_FLAGS, abi, *[a for i in inc for a in ("-isystem", i)], src, "-o", BINDING,
           "-L" + os.path.join(root, "lib"), *BINDING_LIBS,
           "-L" + HERE, "-l:libtokengate.so", "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"binding failed:\n{r.stdout}\n{r.stderr}")
    os.makedirs(BUILD, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(made_for)
    return BINDING


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
