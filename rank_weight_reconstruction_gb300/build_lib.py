"""Builds the sm_103a shared library ``libaq_gb300.so`` in-tree with nvcc.

The translation units are compiled in parallel and linked with the static CUDA runtime;
the driver's tensor-map encoder is resolved at run time, so nothing else is linked. The
serving calls' marshalling module is compiled beside them by the host compiler, where Python's and
torch's headers are at hand; the library itself asks for neither.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG_DIR, "_build")
LIB_PATH = os.path.join(PKG_DIR, "libaq_gb300.so")
# Checked build (tests only): every plain output store checks its index against the output's
# extent and records a violation as AQ_ERR_BOUNDS in the device status word.
DEBUG_BUILD_DIR = os.path.join(PKG_DIR, "_build_debug")
DEBUG_LIB_PATH = os.path.join(PKG_DIR, "libaq_gb300_debug.so")
SOURCES = ["aq_kernels.cu", "aq_decode.cu", "aq_decode2.cu", "aq_decompose.cu", "aq_host.cu", "aq_noalloc.cu",
           "aq_positions.cu", "aq_attention.cu", "aq_attention_tc.cu",
           "aq_verify.cu", "aq_norm.cu", "aq_nvfp4.cu", "aq_scores.cu"]
HEADERS = ["aq_ptx.cuh", "aq_internal.h", "aq_serve.h", "aq_attention.cuh", "aq_positions.cuh"]

# The serving calls' marshalling, a CPython module of host code over torch tensors (see csrc/aq_python.cpp).
MARSHAL_SOURCE = "aq_python.cpp"
MARSHAL_PATH = os.path.join(PKG_DIR, "_marshal.so")

ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", f"-I{INCLUDE}", f"-I{CSRC}"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libaq_gb300.so")


def _newer_than(target: str, sources) -> bool:
    if not os.path.exists(target):
        return False
    files = [os.path.join(CSRC, f) for f in sources] + [os.path.join(INCLUDE, "aq.h"), os.path.abspath(__file__)]
    return all(os.path.getmtime(f) <= os.path.getmtime(target) for f in files)


def up_to_date(lib: str = LIB_PATH) -> bool:
    return _newer_than(lib, SOURCES + HEADERS)


def _marshal_for() -> str:
    """What the marshalling module is built against: this Python's and torch's versions and places."""
    torch = importlib.util.find_spec("torch")
    return " ".join((sys.version.split()[0], sysconfig.get_paths()["include"],
                     importlib.metadata.version("torch") if torch else "-", torch.origin if torch else "-"))


def marshal_up_to_date() -> bool:
    note = MARSHAL_PATH + ".for"
    if not os.path.exists(note) or not _newer_than(MARSHAL_PATH, [MARSHAL_SOURCE]):
        return False
    with open(note) as f:
        return f.read() == _marshal_for()


def _marshal_lacks() -> str | None:
    """What is not there to build the marshalling module with, if anything."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return "torch"
    for need in (os.path.join(sysconfig.get_paths()["include"], "Python.h"),
                 os.path.join(os.path.dirname(spec.origin), "include", "torch", "csrc", "Exceptions.h")):
        if not os.path.exists(need):
            return need
    return None if _host_compiler() else "a host C++ compiler"


def _host_compiler() -> str | None:
    return os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")


def build_marshal(verbose: bool = False) -> str:
    """Compile the marshalling module with the host compiler (needs Python.h and torch's headers)."""
    lacks = _marshal_lacks()
    if lacks:
        raise RuntimeError(f"{lacks} not found: required to build {MARSHAL_PATH}")
    import torch
    include = sysconfig.get_paths()["include"]
    torch_dir = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path()))), "include")
    tmp = MARSHAL_PATH + f".{os.getpid()}.tmp"
    cmd = [_host_compiler(), "-std=c++17", "-O2", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f"-I{include}", f"-I{INCLUDE}",
           *(f"-isystem{d}" for d in (os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"), cuda)),
           os.path.join(CSRC, MARSHAL_SOURCE), "-o", tmp, f"-L{os.path.join(torch_dir, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {MARSHAL_SOURCE}:\n{r.stdout.decode(errors='replace')}")
    os.replace(tmp, MARSHAL_PATH)
    with open(MARSHAL_PATH + ".for", "w") as f:
        f.write(_marshal_for())
    return MARSHAL_PATH


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile (if needed) and return the path of the shared library (the checked build with
    ``debug=True``); the marshalling module too, unless what it needs is not there: the library
    stands without it, and the serving calls of the binding say that it is missing."""
    lib = DEBUG_LIB_PATH if debug else LIB_PATH
    bdir = DEBUG_BUILD_DIR if debug else BUILD_DIR
    stale = force or not marshal_up_to_date()
    lacks = _marshal_lacks() if stale else None
    if lacks:
        print(f"{lacks} not found: {MARSHAL_PATH} is not built", file=sys.stderr)
        if os.path.exists(MARSHAL_PATH):
            os.remove(MARSHAL_PATH)   # of other sources, or of another torch
    if not force and up_to_date(lib):
        if stale and not lacks:
            build_marshal(verbose)
        return lib
    nvcc = nvcc_path()
    os.makedirs(bdir, exist_ok=True)
    procs = []
    for src in SOURCES:
        obj = os.path.join(bdir, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH_FLAGS, *NVCC_FLAGS, *(["-DAQ_DEBUG_CHECKS=1"] if debug else []), "-c",
               os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((src, obj, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    try:
        if stale and not lacks:
            build_marshal(verbose)
    finally:
        outputs = [p.communicate()[0] for _, _, p in procs]
    objs = []
    for (src, obj, p), out in zip(procs, outputs):
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{out.decode(errors='replace')}")
        if verbose and out:
            print(out.decode(errors="replace"), file=sys.stderr)
        objs.append(obj)
    tmp = lib + ".tmp"
    cmd = [nvcc, *ARCH_FLAGS, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout.decode(errors='replace')}")
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv, debug="--debug" in sys.argv))
