"""Compile the layoutmove shared library in place.

Every translation unit under ``csrc/`` -- the host layout algebra, the
copy, tile-copy and exchange planners (plain C++17, compiled with g++) and
the kernels (CUDA, compiled with nvcc for sm_103a only) -- is built in
parallel into ``_build/`` and linked into ``liblayoutmove.so`` next to this
file.  The CUDA runtime is linked
statically, so the library loads without any other CUDA shared object.  The
Python extension ``pycall/lm_pycall.c`` is linked to it as ``_pycall.so``.
"""

from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liblayoutmove.so")
PYCALL_SRC = os.path.join(PKG, "pycall", "lm_pycall.c")
PYCALL = os.path.join(PKG, "_pycall.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC)
                  if f.endswith((".cpp", ".cu")))


def _newest_input() -> float:
    files = _sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                          if f.endswith((".h", ".cuh"))]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files += [os.path.abspath(__file__), PYCALL_SRC]
    return max(os.path.getmtime(f) for f in files)


def build(verbose: bool = False, force: bool = False) -> str:
    """Build (if stale) and return the path of liblayoutmove.so."""
    if (not force and os.path.exists(LIB) and os.path.exists(PYCALL)
            and min(os.path.getmtime(LIB), os.path.getmtime(PYCALL))
            >= _newest_input()):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    common = ["-O3", "-std=c++17", f"-I{INCLUDE}", f"-I{CSRC}"]
    jobs = []
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        if src.endswith(".cu"):
            cmd = [nvcc, *ARCH, "-lineinfo", *common, "-Xcompiler", "-fPIC",
                   "-Xptxas", "-v" if verbose else "-O3",
                   "-c", src, "-o", obj]
        else:
            cmd = [os.environ.get("CXX", "g++"), *common, "-fPIC", "-Wall",
                   "-c", src, "-o", obj]
        jobs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                           stderr=subprocess.STDOUT)))
    failed = []
    for cmd, proc in jobs:
        out, _ = proc.communicate()
        text = out.decode(errors="replace")
        if proc.returncode != 0:
            failed.append(" ".join(cmd) + "\n" + text)
        elif verbose and text.strip():
            sys.stderr.write(text)
    if failed:
        raise RuntimeError("layoutmove build failed:\n" + "\n".join(failed))
    tmp = LIB + ".tmp"
    link = [nvcc, *ARCH, "-shared", "-cudart", "static", *objs, "-o", tmp]
    res = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if res.returncode != 0:
        raise RuntimeError("layoutmove link failed:\n" +
                           res.stdout.decode(errors="replace"))
    os.replace(tmp, LIB)
    tmp = PYCALL + ".tmp"
    link = [os.environ.get("CC", "gcc"), "-O2", "-std=c11", "-Wall", "-shared",
            "-fPIC", f"-I{INCLUDE}", f"-I{sysconfig.get_path('include')}",
            PYCALL_SRC, LIB, "-Wl,-rpath,$ORIGIN", "-o", tmp]
    res = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if res.returncode != 0:
        raise RuntimeError("layoutmove extension failed:\n" +
                           res.stdout.decode(errors="replace"))
    os.replace(tmp, PYCALL)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
