"""Build the IndexCache CUDA library in-tree for sm_100a.

``python -m cross_layer_top_full_b200.build`` (or ``build()``) compiles every
``csrc/*.cu`` with nvcc for ``sm_100a`` and links ``libindexcache.so`` next to
this file.  Objects go to ``_build/`` and are rebuilt only when a source or
header is newer.  Where torch is installed, ``csrc/fastcall.cpp`` becomes
``_fastcall.<tag>.so``: the short way of the quantised-cache calls from Python.
It reads tensors through torch's own inline code, so the tag names the torch and
the Python that it was compiled for, and no others load it.  The calls work
without it, and so does the build.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libindexcache.so")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _newest_header() -> float:
    hs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hs), default=0.0)


def _compile(nvcc: str, src: str, verbose: bool, ptxas_v: bool) -> str:
    obj = os.path.join(OBJDIR, os.path.basename(src) + ".o")
    if (os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(src)
            and os.path.getmtime(obj) >= _newest_header() and not ptxas_v):
        return obj
    cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if ptxas_v:
        cmd += ["-Xptxas", "-v"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0 or (ptxas_v and res.stderr):
        sys.stderr.write(res.stderr)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed on %s" % src)
    return obj


def fast_path() -> str:
    """Path of the short way's module for the torch and the Python that run."""
    import torch
    return os.path.join(PKG, "_fastcall.%s.torch-%s-%s.abi%d.so" % (
        sysconfig.get_config_var("SOABI"), torch.__version__, (torch.version.git_version or "")[:8],
        torch._C._GLIBCXX_USE_CXX11_ABI))


def _build_fastcall(verbose: bool) -> None:
    try:
        import torch
    except ImportError:
        return
    fast = fast_path()
    for old in glob.glob(os.path.join(os.path.dirname(fast), "_fastcall*.so")):
        if old != fast:
            os.remove(old)
    src, header = os.path.join(CSRC, "fastcall.cpp"), os.path.join(INCLUDE, "indexcache.h")
    if os.path.exists(fast) and os.path.getmtime(fast) >= max(os.path.getmtime(src), os.path.getmtime(header)):
        return
    root = os.path.dirname(torch.__file__)
    libs = os.path.join(root, "lib")
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI,
           "-I", INCLUDE, "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I", sysconfig.get_paths()["include"], src, "-o", fast,
           "-L", libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-Wl,-rpath," + libs]
    if verbose:
        print(" ".join(cmd), flush=True)
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
        error = res.stderr if res.returncode else None
    except OSError as e:                                 # no compiler
        error = "%s\n" % e
    if error is not None:
        if os.path.exists(fast):                         # of older sources
            os.remove(fast)
        sys.stderr.write(error + "csrc/fastcall.cpp did not compile: the quantised-cache calls from Python go "
                                 "the long way\n")


def build(verbose: bool = False, ptxas_v: bool = False) -> str:
    """Compile and link the library; returns the path of the .so."""
    os.makedirs(OBJDIR, exist_ok=True)
    nvcc = _nvcc()
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        objs = list(ex.map(lambda s: _compile(nvcc, s, verbose, ptxas_v), srcs))
    if not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs]
        if verbose:
            print(" ".join(cmd), flush=True)
        subprocess.run(cmd, check=True)
    _build_fastcall(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True, ptxas_v="-v" in sys.argv))
