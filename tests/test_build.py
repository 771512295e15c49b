"""The build without a C compiler for the binding's native module, which is optional,
and for more than one interpreter. (A copy of the package's build file; nvcc is a
stand-in that makes empty files.)"""
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PKG = os.path.join(ROOT, "hisparse_top_sparse_gb300")
SUFFIX = sysconfig.get_config_var("EXT_SUFFIX")
NVCC = """#!/bin/sh
echo run >> "$0.log"
while [ $# -gt 0 ]; do [ "$1" = -o ] && : > "$2"; shift; done
"""
RUN = "import _build; stale = _build._stale(); _build.build(); print('stale', stale, 'after', _build._stale())"


@pytest.fixture
def tree(tmp_path):
    os.makedirs(tmp_path / "pkg" / "csrc")
    os.makedirs(tmp_path / "bin")
    shutil.copy(os.path.join(PKG, "_build.py"), tmp_path / "pkg")
    shutil.copy(os.path.join(PKG, "csrc", "hs_call.c"), tmp_path / "pkg" / "csrc")
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    (tmp_path / "pkg" / "csrc" / "a.cu").write_text("")
    nvcc = tmp_path / "bin" / "nvcc"
    nvcc.write_text(NVCC)
    nvcc.chmod(0o755)

    def run(cc):
        env = dict(os.environ, PATH=str(tmp_path / "bin") + os.pathsep + os.environ["PATH"], CC=str(cc))
        return subprocess.run([sys.executable, "-c", RUN], cwd=tmp_path / "pkg", env=env, capture_output=True, text=True,
                              timeout=120)
    run.pkg = tmp_path / "pkg"
    return run


def _modules(pkg):
    return sorted(f for f in os.listdir(pkg) if f.startswith("_call"))


@pytest.mark.parametrize("cc", ["/nonexistent/cc", "/bin/false", "/bin/true", "/bin/sh"])
def test_without_a_compiler_the_library_is_built_all_the_same(tree, cc):
    r = tree(cc)
    assert r.returncode == 0, r.stderr
    assert "stale True after False" in r.stdout and "through ctypes" in r.stderr
    assert os.path.exists(tree.pkg / "libhisparse.so") and _modules(tree.pkg) == []
    # nothing is built again for want of the module
    assert "stale False" in tree(cc).stdout


def test_a_module_is_its_interpreters(tree):
    (tree.pkg / "_call.so").write_text("of another interpreter")
    r = tree("cc")
    assert r.returncode == 0, r.stderr
    assert _modules(tree.pkg) == ["_call" + SUFFIX] and "stale True after False" in r.stdout
    assert not r.stderr
    # a module that no longer compiles does not stay behind
    src = tree.pkg / "csrc" / "hs_call.c"
    src.write_text(src.read_text() + "\n#error\n")
    later = os.path.getmtime(tree.pkg / ("_call" + SUFFIX)) + 10
    os.utime(src, (later, later))
    r = tree("cc")
    assert r.returncode == 0 and _modules(tree.pkg) == [] and "#error" in r.stderr
