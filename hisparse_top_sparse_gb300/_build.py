"""Builds libhisparse.so in-tree from csrc/*.cu for sm_103a with nvcc.

Each translation unit is compiled in parallel, then linked with the static
CUDA runtime into one shared library next to this file.
"""

from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libhisparse.so")
INCLUDE = os.path.join(ROOT, "include")
CALL_SRC = os.path.join(CSRC, "hs_call.c")     # the binding's short way (a Python module)
CALL = os.path.join(HERE, "_call.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libhisparse")


def _no_headers() -> bool:
    """No C headers of this Python: the binding then does without its short way."""
    return not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    if not os.path.exists(LIB) or not (os.path.exists(CALL) or _no_headers()):
        return True
    t = min(os.path.getmtime(p) for p in (LIB, CALL) if os.path.exists(p))
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [
        CALL_SRC, os.path.join(INCLUDE, "hisparse.h"), __file__]
    return any(os.path.getmtime(p) > t for p in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if needed) and return the path of libhisparse.so."""
    if not force and not _stale():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    procs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        objs.append(obj)
        cmd = [nvcc, *ARCH, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                            stderr=subprocess.STDOUT)))
    if not _no_headers():
        cmd = [os.environ.get("CC", "cc"), "-O2", "-fPIC", "-shared", "-I" + sysconfig.get_paths()["include"],
               "-I" + INCLUDE, CALL_SRC, "-o", CALL + ".tmp"]
        procs.append((cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    errors = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            errors.append(" ".join(cmd) + "\n" + out.decode(errors="replace"))
    if errors:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errors))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + res.stdout.decode(errors="replace"))
    os.replace(tmp, LIB)
    if os.path.exists(CALL + ".tmp"):
        os.replace(CALL + ".tmp", CALL)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
