"""Build the CUDA library ``libfh.so`` in-tree for sm_100a (B200), and its Python binding.

Compiles every ``csrc/*.cu`` with nvcc (``-gencode arch=compute_100a,code=sm_100a``)
and links them into ``audio_driven_talking_b200/libfh.so``; compiles ``csrc/bind.cpp`` with
g++ against torch's headers into ``audio_driven_talking_b200/_fhbind.so``. Objects go to
``audio_driven_talking_b200/_build/`` and are rebuilt only when a source or header
is newer. Run ``python -m audio_driven_talking_b200.build`` (or call ``build()``).
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJ = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libfh.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
BIND = os.path.join(PKG, "_fhbind.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))
    return max(os.path.getmtime(h) for h in hs)


def _compile(src: str, extra: list[str], force: bool) -> str:
    obj = os.path.join(OBJ, os.path.basename(src) + ".o")
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), _newest_header()):
        return obj
    cmd = [nvcc(), *ARCH, *FLAGS, *extra, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    if r.stderr.strip():
        sys.stderr.write(r.stderr)
    return obj


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile and link libfh.so; returns its path."""
    os.makedirs(OBJ, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(lambda s: _compile(s, extra, force or verbose_ptxas), srcs))
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < max(os.path.getmtime(o) for o in objs):
        cmd = [nvcc(), *ARCH, "-shared", "-Xlinker", "-soname=libfh.so", "-o", LIB, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    _build_bind(force)
    return LIB


def _bind_made_for() -> str:
    """What the binding module was compiled against besides this project's files."""
    import torch
    return f"{torch.__version__} {torch.version.git_version} {sys.implementation.cache_tag} {os.path.dirname(torch.__file__)}"


def _build_bind(force: bool) -> None:
    """Compile the binding module, which takes its tensors from torch and links to libfh.so. It is rebuilt
    for another torch or Python too: their ABI is not this project's to keep."""
    headers = [os.path.join(INCLUDE, h) for h in ("fh.h", "fh_ops.h")]
    stamp, made_for = os.path.join(OBJ, "bind.made_for"), _bind_made_for()
    if (not force and os.path.exists(BIND) and os.path.exists(stamp) and open(stamp).read() == made_for and
            os.path.getmtime(BIND) >= max(map(os.path.getmtime, [BIND_SRC, *headers]))):
        return
    import sysconfig

    import torch
    troot = os.path.dirname(torch.__file__)
    tinc = os.path.join(troot, "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", tinc, "-isystem", os.path.join(tinc, "torch", "csrc", "api", "include"),
           "-isystem", cuda, "-isystem", sysconfig.get_paths()["include"], BIND_SRC, "-o", BIND,
           "-L", PKG, "-lfh", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(troot, "lib"),
           "-ltorch_python", "-ltorch", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {BIND_SRC}:\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(made_for)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="--ptxas" in sys.argv))
