"""Compile the CUDA library (csrc/*.cu) for sm_103a into libgdn_gb300.so in
this package directory.  Each translation unit compiles in parallel with
nvcc; the objects are then linked into one shared library (static cudart).
The layer operators' direct binding (csrc/binding.cpp, against the installed
PyTorch's headers) becomes _layer_calls.so beside it."""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB_NAME = "libgdn_gb300.so"
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "--expt-relaxed-constexpr", "-I", INCLUDE] + ARCH


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _no_binding(out, why) -> None:
    """The binding is left out, and no older one stays in its place."""
    if os.path.exists(out):
        os.remove(out)
    warnings.warn(f"_layer_calls.so is not built, calls go through ctypes: {why}", RuntimeWarning)


def build_binding() -> str | None:
    """Compile csrc/binding.cpp into _layer_calls.so with the host compiler
    (None, with a warning, where that fails, as it does without Python's
    headers: the binding in Python then makes every call itself)."""
    import torch
    src = os.path.join(CSRC, "binding.cpp")
    out = os.path.join(HERE, "_layer_calls.so")
    if not os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h")):
        return _no_binding(out, "Python.h is missing")
    newest = max(os.path.getmtime(p) for p in
                 [src, torch.__file__] + glob.glob(os.path.join(INCLUDE, "*.h")))
    if os.path.exists(out) and os.path.getmtime(out) >= newest:
        return out
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    libs = os.path.join(root, "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(root, "include"), "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(cuda, "include"), src, "-o", out + ".tmp", "-L", libs,
           "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{libs}"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        return _no_binding(out, str(e))
    if r.returncode != 0:
        return _no_binding(out, f"{cmd[0]} failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(out + ".tmp", out)
    return out


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def build(verbose: bool = False, extra_flags=()) -> str:
    out_dir = os.path.join(HERE, "_build")
    os.makedirs(out_dir, exist_ok=True)
    srcs = sources()
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    newest_dep = max(os.path.getmtime(p) for p in headers + srcs)
    flags = NVCC_FLAGS + list(extra_flags)

    def compile_one(src):
        obj = os.path.join(out_dir, os.path.basename(src) + ".o")
        if os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep:
            return obj
        cmd = [nvcc()] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 4))) as ex:
        binding = ex.submit(build_binding)
        objs = list(ex.map(compile_one, srcs))
        binding.result()
    lib = os.path.join(HERE, LIB_NAME)
    cmd = [nvcc()] + ARCH + ["-shared", "-o", lib + ".tmp"] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(lib + ".tmp", lib)
    return lib


if __name__ == "__main__":
    print(build(verbose=True))
