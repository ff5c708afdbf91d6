"""Build libdelta.so (the C-ABI CUDA library) in-tree for sm_103a.

Each translation unit under ``csrc/`` is compiled by nvcc in parallel, then
linked into ``weight_rnn_gb300/libdelta.so``.  The CUDA runtime is linked
statically and the driver API is reached at run time through
``cudaGetDriverEntryPoint``, so the library loads on a machine without a GPU
(it only fails when asked to compute).

``csrc/binding.cpp``, the Python calls of the block operators' common case, is
compiled by the host compiler against PyTorch's headers and linked to the
library.  Where that fails the package works without it (its calls then go
through ctypes alone, which costs a small call about 10 us more), so a failure
is reported and not raised.

    python -m weight_rnn_gb300.build [--force] [-v]
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libdelta.so")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(PKG, "_fast.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-Wall", "-I", os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"),
                 "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libdelta")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return (sorted(glob.glob(os.path.join(CSRC, "*.cuh")))
            + sorted(glob.glob(os.path.join(CSRC, "*.h")))
            + [os.path.join(ROOT, "include", "delta.h")])


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def binding_command(obj):
    """How to compile binding.cpp, or None where there is nothing to do it with."""
    import sysconfig
    try:
        import torch
    except ImportError:
        return None
    cxx = os.environ.get("CXX") or shutil.which("g++")
    if not cxx:
        return None
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    where = os.path.join(os.path.dirname(torch.__file__), "include")
    return [cxx, "-O2", "-std=c++17", "-fPIC",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I", where, "-I", os.path.join(where, "torch", "csrc", "api", "include"),
            "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
            "-c", BINDING_SRC, "-o", obj]


def binding_made_with():
    """What a built module belongs to besides its sources."""
    import importlib.metadata
    try:
        torch = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch = "none"
    return f"torch {torch}, python {sys.version}, {os.environ.get('CXX') or shutil.which('g++')}"


def _binding_note():
    return os.path.join(BUILD, os.path.basename(BINDING) + ".from")


def _binding_is_stale():
    if _stale(BINDING, [BINDING_SRC, os.path.join(ROOT, "include", "delta.h")]):
        return True
    try:
        with open(_binding_note()) as f:
            return f.read() != binding_made_with()
    except OSError:
        return True


def _discard_binding():
    """A module of other sources or another torch is not to be loaded."""
    for path in (BINDING, _binding_note()):
        if os.path.exists(path):
            os.remove(path)


def link_binding(obj):
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    # torch's libraries are in the process before this one is loaded
    cmd = [os.environ.get("CXX") or shutil.which("g++"), "-shared", "-o", tmp, obj,
           "-L", PKG, "-l:libdelta.so", "-Wl,-rpath,$ORIGIN", "-L", libs, "-ltorch_python",
           "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(r.stdout + r.stderr)
    os.replace(tmp, BINDING)
    with open(_binding_note(), "w") as f:
        f.write(binding_made_with())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link; returns the path of libdelta.so."""
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    hdrs = headers()
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + hdrs):
            cmd = [cc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
            jobs.append(cmd)

    bobj = os.path.join(BUILD, "binding.o")
    bcmd = None
    if force or _binding_is_stale():
        bcmd = binding_command(bobj)
        if bcmd is None:
            _discard_binding()

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    failed = []
    with ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        bjob = ex.submit(run, bcmd) if bcmd else None
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0:
                failed.append(cmd[-3])
    if failed:
        raise RuntimeError(f"nvcc failed for: {failed}")
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(tmp, LIB)
    if bjob is not None:
        r = bjob.result()[1]
        try:
            if r.returncode != 0:
                raise RuntimeError(r.stdout + r.stderr)
            link_binding(bobj)
        except RuntimeError as e:
            _discard_binding()
            sys.stderr.write(f"binding.cpp was not built; calls go through ctypes alone:\n{e}\n")
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-v", "--verbose", action="store_true")
    args = ap.parse_args()
    print(build(force=args.force, verbose=args.verbose))
