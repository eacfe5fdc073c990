"""Builds libnanochat_b200.so in-tree with nvcc for sm_100a.

Also builds _serving.so, the Python binding of the serving calls, against it
(skipped with a message where PyTorch or g++ is absent; nothing else needs it).
Each csrc/*.cu is compiled to an object under _build/ (in parallel, only when
it or a header changed), then all objects are linked into one shared library
next to this file.  Usage: python -m bwd_step_b200.build [--force] [-v]
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libnanochat_b200.so")
SERVING = os.path.join(HERE, "_serving.so")  # Python binding of the serving calls
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
          "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h"))


def _compile(src: str, force: bool, verbose: bool, extra=()):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    newest = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in _headers()])
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj, None
    cmd = [nvcc()] + ARCH + CFLAGS + list(extra) + ["-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, (r.stdout + r.stderr).strip() or None


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(lambda s: _compile(s, force or ptxas_info, verbose, extra), srcs))
    objs = [o for o, _ in results]
    for _, msg in results:
        if msg and (verbose or ptxas_info):
            print(msg)
    newest = max(os.path.getmtime(o) for o in objs)
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        cmd = [nvcc()] + ARCH + ["-shared", "-o", LIB] + objs
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    _build_serving(force, verbose)
    return LIB


def _build_serving(force: bool, verbose: bool):
    """Where the source, a header, PyTorch or Python has changed: the binding uses PyTorch's and Python's internals, so
    one built for others may not load, or load and misread them.  What it was built for stands beside it."""
    import sysconfig
    try:
        import torch
    except ImportError:
        print("serving binding not built: PyTorch is absent", file=sys.stderr)
        return
    cxx = shutil.which("g++")
    if cxx is None:
        print("serving binding not built: g++ is absent", file=sys.stderr)
        return
    src = os.path.join(CSRC, "serving_py.cpp")
    newest = max(os.path.getmtime(f) for f in [src] + glob.glob(os.path.join(INCLUDE, "*.h")))
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    made_for = f"torch {torch.__version__}, C++ ABI {abi}, {sysconfig.get_config_var('SOABI')}\n"
    stamp = SERVING + ".for"
    if not force and os.path.exists(SERVING) and os.path.getmtime(SERVING) >= newest and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == made_for:
                return
    root = os.path.dirname(torch.__file__)
    inc = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"]]
    cmd = [cxx, "-std=c++17", "-O2", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
           "-DUSE_CUDA", *[f"-I{d}" for d in inc], src, "-o", SERVING, f"-L{HERE}", "-lnanochat_b200", "-Wl,-rpath,$ORIGIN",
           f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building {SERVING} failed:\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(made_for)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, ptxas_info="--ptxas" in sys.argv))
