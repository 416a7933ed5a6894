"""Build the sm_103a CUDA library in-tree with nvcc (no cmake; torch only for the binding).

Produces ``libgb300gemm.so`` next to this file from ``csrc/*.cu`` (the GEMM)
and ``csrc/ops/*.cu`` (the operators beside it); the compiled code targets
exactly sm_103a (GB300).  The operators' CPython binding ``_binding*.so``
(``csrc/ops/binding.cpp``) is built against the installed torch; without torch,
or with one that has no CUDA, the library is built alone.
"""
from __future__ import annotations

import glob
import hashlib
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libgb300gemm.so"
LIB_PATH = os.path.join(HERE, LIB_NAME)
BINDING_SRC = os.path.join(CSRC, "ops", "binding.cpp")
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the GB300 GEMM library needs the CUDA toolkit to build")


def _cuda() -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "ops", "*.cu")))


def _inputs():
    return (sources() + sorted(glob.glob(os.path.join(CSRC, "**", "*.cuh"), recursive=True)) +
            sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [os.path.abspath(__file__)])


def _newer(target, inputs) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in inputs)


def _torch():
    """The installed torch's folder and the text of its version.py; None for no
    torch, or one without CUDA (its version.py says cuda = None)."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    folder, version = spec.submodule_search_locations[0], ""
    path = os.path.join(folder, "version.py")
    if os.path.exists(path):
        with open(path, encoding="utf-8") as f:
            version = f.read()
    return None if re.search(r"^cuda\b[^=\n]*=\s*None", version, re.M) else (folder, version)


def binding_path():
    """Where the binding for the installed torch lies, or None without a torch for
    it.  It is compiled against torch's C++ classes, so its name holds a hash of
    which torch that is: another one never loads it."""
    torch = _torch()
    if torch is None:
        return None
    which = hashlib.sha256("\n".join(torch).encode())
    return os.path.join(HERE, "_binding_" + which.hexdigest()[:8] + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))


def up_to_date() -> bool:
    path = binding_path()
    return _newer(LIB_PATH, _inputs()) and (path is None or _newer(path, _binding_inputs()))


def _binding_inputs():
    return [BINDING_SRC, *sorted(glob.glob(os.path.join(INCLUDE, "*.h"))), os.path.abspath(__file__)]


def _build_binding(path):
    """Start compiling the binding; returns (process, its output, command)."""
    tmp = path + f".tmp{os.getpid()}"
    torch, _ = _torch()
    cmd = [os.environ.get("CXX") or shutil.which("g++") or "c++", "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", "-I", sysconfig.get_paths()["include"], "-I", INCLUDE,
           "-isystem", os.path.join(torch, "include"), "-isystem", os.path.join(_cuda(), "include"), BINDING_SRC,
           "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-o", tmp]
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True), tmp, cmd


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library and the binding if any source is newer than them;
    return the library's path."""
    if not force and up_to_date():
        return LIB_PATH
    path = binding_path()
    binding = None
    if path is not None and (force or not _newer(path, _binding_inputs())):
        binding, binding_tmp, binding_cmd = _build_binding(path)
    try:
        if force or not _newer(LIB_PATH, _inputs()):
            _build_library(verbose)
    finally:
        if binding is not None:
            said, _ = binding.communicate()
            if binding.returncode == 0:
                os.replace(binding_tmp, path)
    if binding is not None and binding.returncode != 0:
        raise RuntimeError("the binding failed to build:\n" + " ".join(binding_cmd) + "\n" + said)
    return LIB_PATH


def _build_library(verbose):
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    nvcc = _nvcc()
    # The CUDA runtime is linked shared: with torch in the process both use one
    # runtime (a second, static one slowed every call that follows a torch
    # allocation by about 3 us).
    cudalib = os.path.join(_cuda(), "lib64")
    cmd = [nvcc, *ARCH_FLAGS, "-t", "0", "-O3", "-lineinfo", "-std=c++17",
           "-Xcompiler", "-fPIC,-fvisibility=hidden", "-shared",
           "-cudart", "shared", "-Xlinker", "-rpath," + cudalib, "-I", INCLUDE, "-I", CSRC, *sources(), "-o", tmp]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + res.stdout + res.stderr)
    if verbose:
        print(res.stdout + res.stderr)
    os.replace(tmp, LIB_PATH)
