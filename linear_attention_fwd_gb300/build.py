"""Build libkda.so in-tree for sm_103a (nvcc, no cmake), and _binding.so, the C++ side of the Python
binding, with the host compiler.  The library needs neither Python's headers nor PyTorch: where the binding
cannot be built, build() warns and returns the library all the same (build_binding() raises).

Each .cu under csrc/ compiles to its own object in parallel; the objects link
into ``libkda.so`` beside this file.  The CUDA runtime is linked statically and
the driver API is reached through ``cudaGetDriverEntryPointByVersion``, so the
library loads on a machine without a GPU driver (it only needs one to run).
"""
from __future__ import annotations

import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkda.so")
LIB_DEBUG = os.path.join(HERE, "libkda_debug.so")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_STAMP = os.path.join(BUILD, "stamp_binding")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-v"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    hs += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    return sorted(hs)


def _digest(paths, extra=""):
    h = hashlib.sha256(extra.encode())
    for p in paths:
        h.update(p.encode())
        with open(p, "rb") as f:
            h.update(f.read())
    return h.hexdigest()


def build_binding(force: bool = False) -> str:
    """Compile csrc/binding.cpp against the installed PyTorch into _binding.so; returns its path.  Raises
    where that fails; a _binding.so of other sources is then removed (it may not fit the library)."""
    import torch
    src = os.path.join(CSRC, "binding.cpp")
    root = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    flags = ["-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"), cuda]
    libs = ["torch_python", "torch_cuda", "torch_cpu", "c10_cuda", "c10"]
    want = _digest([src, os.path.join(INCLUDE, "kda.h")], " ".join(flags + inc + [torch.__version__, sys.version]))
    os.makedirs(os.path.dirname(BINDING_STAMP), exist_ok=True)
    if not force and os.path.exists(BINDING) and os.path.exists(BINDING_STAMP):
        with open(BINDING_STAMP) as f:
            if f.read() == want:
                return BINDING
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), *flags, *(f"-I{i}" for i in inc), src, "-o", tmp,
           f"-L{os.path.join(root, 'lib')}", *(f"-l{x}" for x in libs)]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{cmd[0]} failed for {src}:\n{r.stdout}\n{r.stderr}")
    except (OSError, RuntimeError):
        for old in (BINDING_STAMP, BINDING):
            if os.path.exists(old):
                os.remove(old)
        raise
    os.replace(tmp, BINDING)
    with open(BINDING_STAMP, "w") as f:
        f.write(want)
    return BINDING


def build(verbose: bool = False, force: bool = False, debug: bool = False) -> str:
    """Compile csrc/*.cu for sm_103a and link libkda.so (and build _binding.so beside it, warning where
    that cannot be done); returns the library's path.

    debug=True builds libkda_debug.so instead (objects in _build_debug/): the same kernels with
    KDA_DEBUG_CHECKS defined, so that every chunk forward and decode call first checks the log decays
    and the packed offsets on the device (kda_debug_checks, kda_device_status)."""
    build_dir = BUILD + "_debug" if debug else BUILD
    lib_path = LIB_DEBUG if debug else LIB
    flags = NVCC_FLAGS + (["-DKDA_DEBUG_CHECKS=1"] if debug else [])
    os.makedirs(build_dir, exist_ok=True)
    nvcc = _nvcc()
    srcs = _sources()
    hdr_digest = _digest(_headers(), " ".join(ARCH + flags))
    stamp = os.path.join(build_dir, "stamp")
    want = _digest(srcs, hdr_digest)
    with ThreadPoolExecutor(max_workers=1) as side:   # beside the kernels
        binding = side.submit(build_binding, force)
        path = _build_library(verbose, force, build_dir, lib_path, flags, nvcc, srcs, stamp, want)
        failed = binding.exception()
    if failed is not None:
        warnings.warn(f"{os.path.basename(path)} is built, {os.path.basename(BINDING)} is not; the calls bound through it "
                      f"(linear attention, paged cache) raise from Python: {failed}", RuntimeWarning, stacklevel=2)
    return path


def _build_library(verbose, force, build_dir, lib_path, flags, nvcc, srcs, stamp, want) -> str:
    if not force and os.path.exists(lib_path) and os.path.exists(stamp):
        with open(stamp) as f:
            if f.read() == want:
                return lib_path

    def compile_one(src):
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *ARCH, *flags, "-I", INCLUDE, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        with open(obj + ".log", "w") as f:
            f.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = list(ex.map(compile_one, srcs))
    tmp = lib_path + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)
    with open(stamp, "w") as f:
        f.write(want)
    if verbose:
        for o in objs:
            with open(o + ".log") as f:
                sys.stdout.write(f.read())
    return lib_path


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv, force="-f" in sys.argv, debug="--debug" in sys.argv))
