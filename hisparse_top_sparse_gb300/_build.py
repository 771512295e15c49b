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
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libhisparse.so")
INCLUDE = os.path.join(ROOT, "include")
CALL_SRC = os.path.join(CSRC, "hs_call.c")     # the binding's short way (a Python module)
# (tagged with the interpreter whose object layouts it was compiled against: no other loads it)
CALL = os.path.join(HERE, "_call" + sysconfig.get_config_var("EXT_SUFFIX"))
NO_CALL = os.path.join(BUILD, os.path.basename(CALL) + ".failed")    # why there is none

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is needed to build libhisparse")


def _start_call(verbose: bool):
    """(what compiles the binding's short way, None) or (None, why nothing does): the
    binding can do without it."""
    include = sysconfig.get_paths()["include"]
    if not os.path.exists(os.path.join(include, "Python.h")):
        return None, "no Python.h in " + include
    cmd = [os.environ.get("CC", "cc"), "-O2", "-fPIC", "-shared", "-I" + include, "-I" + INCLUDE, CALL_SRC,
           "-o", CALL + ".tmp"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    if os.path.exists(CALL + ".tmp"):
        os.remove(CALL + ".tmp")
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT), None
    except OSError as e:
        return None, str(e)


def _wait_call(proc, why):
    """Why there is no module, None where there is one."""
    if proc is not None:
        out, _ = proc.communicate()
        if proc.returncode != 0 or not os.path.exists(CALL + ".tmp"):
            why = " ".join(proc.args) + "\n" + out.decode(errors="replace")
    return why


def _place_call(why) -> None:
    """Puts the module in its place, or notes and says why there is none."""
    for path in (NO_CALL, os.path.join(HERE, "_call.so"), *((CALL, CALL + ".tmp") if why else ())):
        if os.path.exists(path):       # (an untagged module is an earlier version's)
            os.remove(path)
    if why:
        with open(NO_CALL, "w") as f:
            f.write(why + "\n")
        warnings.warn("the binding's native module is not built, its calls go through ctypes: " + why)
    else:
        os.replace(CALL + ".tmp", CALL)


def sources() -> list:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale() -> bool:
    call = CALL if os.path.exists(CALL) else NO_CALL
    if not os.path.exists(LIB) or not os.path.exists(call):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(call))
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
    call, no_call = _start_call(verbose)
    errors = []
    for cmd, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            errors.append(" ".join(cmd) + "\n" + out.decode(errors="replace"))
    no_call = _wait_call(call, no_call)
    if errors:
        raise RuntimeError("nvcc failed:\n" + "\n".join(errors))
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs]
    res = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n" + res.stdout.decode(errors="replace"))
    os.replace(tmp, LIB)
    _place_call(no_call)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
