"""Build libpagedattn.so in-tree for sm_100a.

    python -m paged_kv_cache_350_b200.build [--force] [-v]

Compiles every source under ``csrc/`` with nvcc (``-gencode
arch=compute_100a,code=sm_100a -lineinfo -O3``), links one shared library with
the CUDA runtime linked statically, and places it next to this file, where the
Python binding loads it.  ``_calls.so``, the Python module with the step calls on torch
tensors, is compiled beside it with the host compiler against the installed torch (without one it is left
out).  Objects go to ``_build/`` at the repository root.
Rebuilds only what changed unless ``--force``.
"""

from __future__ import annotations

import argparse
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libpagedattn.so")
CALLS = os.path.join(PKG, "_calls.so")  # the step calls on torch tensors (csrc/calls.cpp)
CALLS_STAMP = os.path.join(BUILD, "_calls.made_for")

SOURCES = ["api.cu", "decode_tc.cu", "decode_stream.cu", "decode_generic.cu", "cache_ops.cu", "allocator.cpp",
           "decode_noalloc.cu", "decode_prefix.cu", "selftest.cu", "pipeline.cpp",
           "rope.cu", "attention.cu", "attention_tc.cu", "attention_tokens.cu",
           "attention_tokens32.cu", "beam.cu", "api_ops.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC]


def nvcc():
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libpagedattn")
    return path


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return hs + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force=False, verbose=False, extra_flags=(), out=None, build_dir=None):
    """Compile and link; ``out``/``build_dir`` place a variant build elsewhere."""
    lib_path = out or LIB
    bdir = build_dir or BUILD
    os.makedirs(bdir, exist_ok=True)
    headers = _headers()
    cc = nvcc()
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(bdir, src + ".o")
        objs.append(o)
        if force or _stale(o, [s] + headers):
            cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", s, "-o", o]
            if src.endswith(".cu"):
                cmd += ["-Xptxas", "-v"] if verbose else []
            jobs.append(cmd)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with ThreadPoolExecutor(max(1, min(len(jobs), os.cpu_count() or 1))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode:
                raise RuntimeError(f"nvcc failed on {cmd[-3]}")
    if force or jobs or _stale(lib_path, objs):
        tmp = lib_path + ".tmp"
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("linking libpagedattn.so failed")
        os.replace(tmp, lib_path)
    if out is None:
        build_calls(force=force, verbose=verbose)
    return lib_path


def _calls_made_for():
    """The torch and the Python that _calls.so is built against (None without torch); imports neither."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return None
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:  # (not an installed package: a tree on the path)
        version = str(os.path.getmtime(spec.origin))
    return "\n".join([version, spec.origin, sys.version])


def calls_stale():
    """Whether _calls.so is older than its sources, or made for another torch or Python."""
    if _stale(CALLS, [os.path.join(CSRC, "calls.cpp"), os.path.join(INCLUDE, "pa.h")]):
        return True
    try:
        with open(CALLS_STAMP) as f:
            return f.read() != _calls_made_for()
    except FileNotFoundError:
        return True


def build_calls(force=False, verbose=False):
    """The Python extension module with the step calls: host code against torch's headers."""
    src = os.path.join(CSRC, "calls.cpp")
    made_for = _calls_made_for()
    if made_for is None:
        sys.stderr.write("torch is not installed: the step calls (_calls.so) are not built\n")
        return None
    if not force and not calls_stale():
        return CALLS
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    lib = os.path.join(root, "lib")
    tmp = CALLS + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"], src, "-o", tmp,
           "-L", lib, f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if verbose or r.returncode:
        sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode:
        raise RuntimeError("compiling _calls.so failed")
    os.replace(tmp, CALLS)
    os.makedirs(BUILD, exist_ok=True)
    with open(CALLS_STAMP, "w") as f:
        f.write(made_for)
    return CALLS


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    a = ap.parse_args(argv)
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()
