"""In-tree build of libnats.so with nvcc for sm_103a (no cmake, no torch), and
of _operators.so, the operators' torch-facing binding, with g++.

Each translation unit under csrc/ compiles in parallel to an object under
_build/, then the two shared libraries are linked next to this file.  libnats.so
needs neither torch nor Python: it is built also where the binding cannot be.
"""

from __future__ import annotations

import fcntl
import glob
import importlib.metadata
import os
import platform
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libnats.so")
BINDING = os.path.join(PKG, "_operators.so")
STAMP = os.path.join(BUILD, "binding.txt")  # what the binding was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
    "-I" + os.path.join(ROOT, "include"),
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _binding_source():
    return os.path.join(CSRC, "binding.cpp")


def _lib_deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + [
        os.path.join(ROOT, "include", "nats.h"), os.path.abspath(__file__)]


def _binding_deps():
    return [_binding_source(), os.path.join(ROOT, "include", "nats.h"), os.path.abspath(__file__)]


def _abi() -> str:
    """What a built binding goes with: this Python and this torch."""
    try:
        torch_version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        torch_version = "none"
    return f"python {sys.version}, torch {torch_version}, {platform.machine()}"


def _newer(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(p) <= os.path.getmtime(path) for p in deps)


def _lib_up_to_date() -> bool:
    return _newer(LIB, _lib_deps())


def _binding_up_to_date() -> bool:
    if not _newer(BINDING, _binding_deps()) or not os.path.exists(STAMP):
        return False
    with open(STAMP) as f:
        return f.read() == _abi()


def up_to_date() -> bool:
    return _lib_up_to_date() and _binding_up_to_date()


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile libnats.so and _operators.so where a source, or for the second Python or torch, has changed; returns
    the first one's path.  A failure of the second leaves the first one built.

    Serialised across processes with a file lock (several ranks may call it)."""
    if not force and up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with open(os.path.join(BUILD, ".lock"), "w") as lk:
        fcntl.flock(lk, fcntl.LOCK_EX)
        try:
            if not force and up_to_date():
                return LIB
            return _build_locked(force, verbose, extra_flags)
        finally:
            fcntl.flock(lk, fcntl.LOCK_UN)


def _build_binding(verbose) -> None:
    """_operators.so: one file against Python's and torch's headers, linked to torch's own libraries."""
    import torch

    root = os.path.dirname(torch.__file__)
    libs = os.path.join(root, "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           "-isystem", os.path.join(root, "include"),
           "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include"),
           "-I" + os.path.join(ROOT, "include"), _binding_source(), "-o", tmp, "-L" + libs, "-Wl,-rpath," + libs,
           "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    with open(STAMP, "w") as f:
        f.write(_abi())


def _build_lib(ex, verbose, extra_flags) -> None:
    nvcc = _nvcc()
    srcs = _sources()
    objs = [os.path.join(BUILD, os.path.basename(s)[:-3] + ".o") for s in srcs]

    def compile_one(args):
        src, obj = args
        cmd = [nvcc] + NVCC_FLAGS + list(extra_flags) + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stderr.strip() or r.stdout.strip()):
            print(r.stdout + r.stderr, flush=True)
        return obj

    list(ex.map(compile_one, zip(srcs, objs)))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def _build_locked(force, verbose, extra_flags) -> str:
    with ThreadPoolExecutor(max_workers=max(1, min(len(_sources()) + 1, os.cpu_count() or 4))) as ex:
        binding = None if _binding_up_to_date() and not force else ex.submit(_build_binding, verbose)
        if force or not _lib_up_to_date():
            _build_lib(ex, verbose, extra_flags)
        if binding is not None:
            try:
                binding.result()
            except Exception as e:
                raise RuntimeError(f"libnats.so is built, its torch binding is not: {e}") from e
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
