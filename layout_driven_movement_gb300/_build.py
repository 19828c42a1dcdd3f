"""Compile the layoutmove shared library in place.

Every translation unit under ``csrc/`` -- the host layout algebra, the
copy, tile-copy and exchange planners (plain C++17, compiled with g++) and
the kernels (CUDA, compiled with nvcc for sm_103a only) -- is built in
parallel into ``_build/`` and linked into ``liblayoutmove.so`` next to this
file.  The CUDA runtime is linked
statically, so the library loads without any other CUDA shared object.  The
Python extension ``pycall/lm_pycall.c`` is linked to it as ``_pycall`` with
the interpreter's own suffix.  It alone needs Python's headers: where it cannot
be built the library still is, and the calls that go through it say why they
cannot be made.
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
PYCALL = os.path.join(PKG, "_pycall" + sysconfig.get_config_var("EXT_SUFFIX"))
PYCALL_LOG = os.path.join(BUILD, "pycall.log")

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
    files.append(os.path.abspath(__file__))
    return max(os.path.getmtime(f) for f in files)


def build(verbose: bool = False, force: bool = False) -> str:
    """Build what is stale; return the path of liblayoutmove.so."""
    os.makedirs(BUILD, exist_ok=True)
    if (force or not os.path.exists(LIB)
            or os.path.getmtime(LIB) < _newest_input()):
        _build_library(verbose)
    if (force or not os.path.exists(PYCALL) or os.path.getmtime(PYCALL)
            < max(os.path.getmtime(f) for f in (LIB, PYCALL_SRC))):
        _build_extension()
    return LIB


def _build_library(verbose: bool) -> None:
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
    # (by its name alone, so that what is linked to it finds the one beside it)
    link = [nvcc, *ARCH, "-shared", "-cudart", "static", "-Xlinker",
            "-soname=" + os.path.basename(LIB), *objs, "-o", tmp]
    res = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if res.returncode != 0:
        raise RuntimeError("layoutmove link failed:\n" +
                           res.stdout.decode(errors="replace"))
    os.replace(tmp, LIB)


def _build_extension() -> None:
    """Links the extension to the library as it is now; where that fails, none
    is left and the log tells why."""
    tmp = PYCALL + ".tmp"
    link = [os.environ.get("CC", "gcc"), "-O2", "-std=c11", "-Wall", "-shared",
            "-fPIC", f"-I{INCLUDE}", f"-I{sysconfig.get_path('include')}",
            PYCALL_SRC, LIB, "-Wl,-rpath,$ORIGIN", "-o", tmp]
    try:
        res = subprocess.run(link, stdout=subprocess.PIPE,
                             stderr=subprocess.STDOUT)
        text, ok = res.stdout.decode(errors="replace"), res.returncode == 0
    except OSError as e:
        text, ok = str(e), False
    with open(PYCALL_LOG, "w") as f:
        f.write(text)
    if ok:
        os.replace(tmp, PYCALL)
        return
    if os.path.exists(PYCALL):
        os.remove(PYCALL)
    sys.stderr.write("layoutmove: the Python extension was not built (rope, "
                     "kv_write, kv_read and kv_attend need it):\n" + text)


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv))
