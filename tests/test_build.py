"""What build() compiles and when, with stand-ins for the compilers (each writes
its output file and a line to a log) on a copy of the package."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = "dense_fp16_gemm_04_gb300"
COMPILER = """#!/bin/sh
echo {name} >> {log}
while [ "$1" != -o ]; do shift; done
echo {name} > "$2"
"""


@pytest.fixture
def tree(tmp_path):
    """A copy of the package's sources; run(code, ...) runs Python there and
    returns the compilers it called."""
    for d in (PACKAGE, "include"):
        shutil.copytree(os.path.join(ROOT, d), tmp_path / d,
                        ignore=shutil.ignore_patterns("*.so", "__pycache__", "*.tmp*"))
    log = tmp_path / "log"
    for name in ("nvcc", "cxx"):
        path = tmp_path / name
        path.write_text(COMPILER.format(name=name, log=log))
        path.chmod(0o755)

    def run(code, cxx="cxx", fails=False, **env):
        log.write_text("")
        r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                           env=dict(os.environ, NVCC=str(tmp_path / "nvcc"), CXX=shutil.which(cxx) or str(tmp_path / cxx), **env))
        assert (r.returncode != 0) == fails, r.stderr
        run.stderr = r.stderr
        return sorted(log.read_text().split())

    run.path = tmp_path
    return run


BUILD = f"import {PACKAGE} as g; g.build()"
NO_TORCH = "import sys; sys.modules['torch'] = None; "


def test_without_torch_the_library_is_built_alone(tree):
    assert tree(NO_TORCH + BUILD) == ["nvcc"]
    assert (tree.path / PACKAGE / "libgb300gemm.so").read_text() == "nvcc\n"
    assert tree(NO_TORCH + BUILD) == []  # up to date


def test_with_torch_the_binding_is_built_too(tree):
    assert tree(BUILD) == ["cxx", "nvcc"]
    assert tree(BUILD) == []


def test_a_failed_binding_leaves_the_library(tree):
    """A finished library is kept when the binding does not compile, and is not
    compiled again for the next try."""
    assert tree(BUILD, cxx="false", fails=True) == ["nvcc"]
    assert "the binding failed to build" in tree.stderr
    assert (tree.path / PACKAGE / "libgb300gemm.so").exists()
    assert tree(BUILD) == ["cxx"]
    assert tree(BUILD) == []


def test_a_failed_library_leaves_the_binding(tree):
    (tree.path / "nvcc").write_text("#!/bin/sh\necho nvcc >> %s\nexit 1\n" % (tree.path / "log"))
    assert tree(BUILD, fails=True) == ["cxx", "nvcc"]
    assert "nvcc failed" in tree.stderr
    assert not (tree.path / PACKAGE / "libgb300gemm.so").exists()
    (tree.path / "nvcc").write_text(COMPILER.format(name="nvcc", log=tree.path / "log"))
    assert tree(BUILD) == ["nvcc"]


def test_another_torch_gets_a_binding_of_its_own(tree):
    """A binding is compiled against one torch's classes: after an upgrade in
    place, or from another folder, it is built again and the old one not loaded."""
    torch = tree.path / "site" / "torch"
    torch.mkdir(parents=True)
    (torch / "__init__.py").write_text("")
    (torch / "version.py").write_text("__version__ = '1'\n")
    old = os.path.getmtime(os.path.join(ROOT, "README.md"))
    env = dict(PYTHONPATH=str(tree.path / "site"))
    assert tree(BUILD, **env) == ["cxx", "nvcc"] and tree(BUILD, **env) == []
    (torch / "version.py").write_text("__version__ = '2'\n")
    os.utime(torch / "version.py", (old, old))  # an installer may keep the files' own dates
    assert tree(BUILD, **env) == ["cxx"] and tree(BUILD, **env) == []
    assert tree(BUILD) == ["cxx"]  # the installed one
    assert len(list((tree.path / PACKAGE).glob("_binding_*.so"))) == 3


def test_star_import(tree):
    """Without torch the GEMM's names; with it the operators' too, torch being
    loaded when one of them is first looked up."""
    star = f"from {PACKAGE} import *; assert gemm and Plan"
    assert tree(NO_TORCH + star + "; assert 'gated_ffn' not in dir()") == []
    assert tree(star + "; assert gated_ffn and w4_linear and orthogonalize") == []
    assert tree(f"import sys, {PACKAGE} as g; assert 'torch' not in sys.modules; assert 'Ops' in g.__all__") == []


def test_a_torch_without_cuda_leaves_the_binding_out(tree):
    """The binding links torch's CUDA library; the GEMM does without."""
    torch = tree.path / "site" / "torch"
    torch.mkdir(parents=True)
    (torch / "__init__.py").write_text("")
    (torch / "version.py").write_text("from typing import Optional\n\n__version__ = '2+cpu'\ncuda: Optional[str] = None\n")
    env = dict(PYTHONPATH=str(tree.path / "site"))
    assert tree(BUILD, **env) == ["nvcc"] and tree(BUILD, **env) == []
    (torch / "version.py").write_text("__version__ = '2+cu130'\ncuda: Optional[str] = '13.0'\nhip: Optional[str] = None\n")
    assert tree(BUILD, **env) == ["cxx"]
