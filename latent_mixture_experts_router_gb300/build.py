"""Compile the CUDA library in-tree: csrc/*.cu -> liblatent_moe.so (sm_103a only).

Each translation unit compiles in its own nvcc process, in parallel; objects go
to ``_build/`` next to this file.  A unit is recompiled when it or any header
under csrc/ or include/ is newer than its object.

The binding's extension _tensors.*.so (csrc/tensors.cpp, torch's and Python's headers, no CUDA) is compiled beside them by
the host compiler, and again where torch, Python or the command are others: it reads torch's objects as those headers lay
them out.  Where that fails the library is made all the same, before build() raises: only the calls that need
the extension are missing then.

``build(checked=True)`` makes the checked variant liblatent_moe_checked.so (objects
in ``_build_checked/``): the same sources with -DLMOE_BOUNDS_CHECKS=1, whose forward
validates the routing structures before any kernel indexes with them.  It is off by
default; the tests that exercise it build it on demand.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "liblatent_moe.so")
LIB_TENSORS = os.path.join(PKG, "_tensors" + sysconfig.get_config_var("EXT_SUFFIX"))   # (with Python's ABI)
BUILD_CHECKED = os.path.join(PKG, "_build_checked")
LIB_CHECKED = os.path.join(PKG, "liblatent_moe_checked.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _cuda_lib_dirs():
    dirs = []
    for d in ("/usr/local/cuda/lib64", "/usr/local/cuda/lib64/stubs",
              "/usr/local/cuda/targets/sbsa-linux/lib", "/usr/local/cuda/targets/sbsa-linux/lib/stubs",
              "/usr/local/cuda/targets/x86_64-linux/lib", "/usr/local/cuda/targets/x86_64-linux/lib/stubs"):
        if os.path.isdir(d):
            dirs.append("-L" + d)
    return dirs


def _torch() -> tuple:
    """torch's directory and version (torch is found, not imported)."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    root = list(spec.submodule_search_locations)[0]
    with open(os.path.join(root, "version.py")) as f:
        return root, re.search(r"__version__ = ['\"]([^'\"]+)", f.read()).group(1)


def _tensors_cmd(src: str) -> list:
    """The host compiler's command for the binding's extension."""
    root, version = _torch()
    inc, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", f'-DLMOE_TORCH_VERSION="{version}"',
            "-I" + sysconfig.get_paths()["include"], "-I" + inc, "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
            src, "-L" + lib, "-ltorch_python", "-ltorch_cpu", "-lc10"]


def _newer(src: str, obj: str, deps) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return os.path.getmtime(src) > t or any(os.path.getmtime(d) > t for d in deps)


def _build_tensors(verbose: bool):
    """The binding's extension, if its source is newer or it was made by another command (for another torch)."""
    src = os.path.join(CSRC, "tensors.cpp")
    cmd = _tensors_cmd(src)
    key, path = "\n".join(cmd), LIB_TENSORS + ".key"
    if os.path.exists(path) and not _newer(src, LIB_TENSORS, ()):
        with open(path) as f:
            if f.read() == key:
                return
    made = LIB_TENSORS + ".new"
    try:
        r = subprocess.run([*cmd, "-o", made], capture_output=True, text=True)
    except OSError as e:   # no compiler
        raise RuntimeError(f"{src}: {e}") from None
    if verbose or r.returncode != 0:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {src}")
    os.replace(made, LIB_TENSORS)
    with open(path, "w") as f:
        f.write(key)


def build(verbose: bool = False, extra_flags=(), checked: bool = False) -> str:
    """Build (or reuse) the shared library and return its path (checked: the bounds-checked
    variant)."""
    BUILD = BUILD_CHECKED if checked else globals()["BUILD"]
    LIB = LIB_CHECKED if checked else globals()["LIB"]
    if checked:
        extra_flags = tuple(extra_flags) + ("-DLMOE_BOUNDS_CHECKS=1",)
    os.makedirs(BUILD, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    deps = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))
    nvcc = _nvcc()
    jobs = []
    for s in srcs:
        obj = os.path.join(BUILD, os.path.basename(s) + ".o")
        if _newer(s, obj, deps):
            jobs.append([nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", obj])
    objs = [os.path.join(BUILD, os.path.basename(s) + ".o") for s in srcs]
    link = bool(jobs)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 1))) as ex:
        extension = None if checked else ex.submit(_build_tensors, verbose)
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed on {cmd[-3]}")
    if link or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        cmd = [nvcc, *ARCH, "-shared", "-o", LIB, *objs, *_cuda_lib_dirs(), "-lcudart"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("link failed")
    if extension is not None:
        extension.result()
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
