"""Build libmoe_gb300.so in-tree with nvcc for sm_103a, and the holders' extension with g++.

    python -m mixture_experts_decode_router_gb300.build

Each ``csrc/*.cu`` is compiled to an object in parallel, then linked into
``_build/libmoe_gb300.so`` (the CUDA runtime linked statically).  No cmake.

The library needs nvcc alone.  ``_build/_moe_torch.so``, through which the Python holders call it
with torch tensors, needs torch, g++ and Python's headers too, and is built when these holders
are first used, or beside the library by ``build_all`` (and the command above).
"""

from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmoe_gb300.so")
EXT = os.path.join(BUILD, "_moe_torch.so")       # the holders' calls on torch tensors
EXT_SRC = os.path.join(CSRC, "moe_torch.cpp")
HEADER = os.path.join(os.path.dirname(PKG), "include", "moe.h")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _compile(nvcc, src, verbose_ptxas=False):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
    if verbose_ptxas:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _compile_ext() -> None:
    import torch
    home, cuda = os.path.dirname(torch.__file__), os.path.dirname(os.path.dirname(_nvcc()))
    inc = [os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           EXT_SRC, "-o", EXT + ".tmp", *("-I" + i for i in inc), "-L" + os.path.join(home, "lib"),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {EXT_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(EXT + ".tmp", EXT)


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")]
    deps.append(HEADER)
    return any(os.path.getmtime(d) > t for d in deps if os.path.exists(d))


def _ext_stale() -> bool:
    if not os.path.exists(EXT):
        return True
    t = os.path.getmtime(EXT)
    return any(os.path.getmtime(d) > t for d in (EXT_SRC, HEADER))


def build_ext(force: bool = False) -> str:
    """Compile the holders' extension (if stale) and return its path; raises without torch."""
    if force or _ext_stale():
        os.makedirs(BUILD, exist_ok=True)
        _compile_ext()
    return EXT


def build_all(force: bool = False, verbose_ptxas: bool = False) -> str:
    """The library and the extension, at the same time."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        ext = ex.submit(build_ext, force)
        lib = build(force, verbose_ptxas)
        ext.result()
    return lib


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile (if stale) and return the path of the shared library (without the extension)."""
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = sources()
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        results = list(ex.map(lambda s: _compile(nvcc, s, verbose_ptxas), srcs))
    objs = [o for o, _ in results]
    if verbose_ptxas:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + ".tmp"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    todo = build_all if importlib.util.find_spec("torch") else build   # (the library alone without torch)
    print(todo(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
