"""Build libgdn.so (the CUDA kernels + C ABI) in-tree for sm_103a.

Each translation unit under csrc/ is compiled by nvcc in parallel, then
linked into ``gated_delta_rule_chunk_gb300/libgdn.so`` with the CUDA runtime
linked statically. ptxas resource usage (registers, spills, shared memory) of
every kernel is written to ``_build/ptxas.log``.

    python -m gated_delta_rule_chunk_gb300.build
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdn.so")
# The GDN_DEBUG build: the same sources with device-side index checks (see gdn_debug_build
# in include/gdn.h), for the tests; the product path loads LIB.
BUILD_DEBUG = os.path.join(PKG, "_build_debug")
LIB_DEBUG = os.path.join(PKG, "libgdn_debug.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgdn")


# The attention calls' marshalling (csrc/attn_torch.cpp), a CPython module over torch's C++ API.
MODULE = os.path.join(PKG, "_attn_torch.so")
MODULE_STAMP = os.path.join(BUILD, "attn_torch.abi")  # module_abi() of the one that is there
MODULE_SRC = os.path.join(CSRC, "attn_torch.cpp")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh"))) + [
        os.path.join(PKG, "..", "include", "gdn.h"),
        os.path.join(PKG, "..", "include", "gdn_attn.h"), os.path.abspath(__file__)]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(p) <= t for p in _deps())


def _compile(src: str, debug: bool = False) -> tuple[str, str]:
    obj = os.path.join(BUILD_DEBUG if debug else BUILD, os.path.basename(src)[:-3] + ".o")
    cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *(["-DGDN_DEBUG"] if debug else []), "-c", src,
           "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stdout + r.stderr


def module_abi() -> str:
    """What the module is built against: one torch and one Python. Empty without torch."""
    try:
        import torch
    except ImportError:
        return ""
    return (f"torch {torch.__version__} in {os.path.dirname(torch.__file__)}, "
            f"{sysconfig.get_config_var('SOABI')}")


def module_built_for() -> str:
    """The module_abi() of the module that is there; empty where that is not known."""
    try:
        with open(MODULE_STAMP) as f:
            return f.read() if os.path.exists(MODULE) else ""
    except OSError:
        return ""


def module_up_to_date() -> bool:
    if not os.path.exists(MODULE) or module_built_for() != module_abi():
        return False
    deps = [MODULE_SRC, os.path.join(PKG, "..", "include", "gdn.h"),
            os.path.join(PKG, "..", "include", "gdn_attn.h"), os.path.abspath(__file__)]
    t = os.path.getmtime(MODULE)
    return all(os.path.getmtime(p) <= t for p in deps)


def build_module() -> str:
    """Compile _attn_torch.so with the host compiler. Returns its path, or an empty string where
    torch or Python's headers are missing: then there is nothing to call it from, and the library
    is complete without it."""
    abi = module_abi()
    python = sysconfig.get_paths()["include"]
    missing = "torch" if not abi else "" if os.path.exists(os.path.join(python, "Python.h")) else "Python.h"
    if missing:
        print(f"{missing} not found: {os.path.basename(MODULE)} (the attention calls from Python) "
              "is not built", file=sys.stderr)
        return ""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = MODULE + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           f"-I{root}/include", f"-I{root}/include/torch/csrc/api/include", f"-I{cuda}/include",
           f"-I{python}", MODULE_SRC, "-o", tmp, f"-L{root}/lib",
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {MODULE_SRC}:\n{r.stdout}\n{r.stderr}")
    os.makedirs(os.path.dirname(MODULE_STAMP), exist_ok=True)
    if os.path.exists(MODULE_STAMP):
        os.remove(MODULE_STAMP)
    os.replace(tmp, MODULE)
    with open(MODULE_STAMP, "w") as f:
        f.write(abi)
    return MODULE


def build(force: bool = False, verbose: bool = False, debug: bool = False) -> str:
    """Compile libgdn.so (libgdn_debug.so with debug=True), and beside it _attn_torch.so,
    unless they are newer than their sources. Returns the library's path; where the module does
    not compile, it raises with the library built."""
    lib, bdir = (LIB_DEBUG, BUILD_DEBUG) if debug else (LIB, BUILD)
    module = not debug and (force or not module_up_to_date())
    if not force and up_to_date(lib):
        if module:
            build_module()
        return lib
    os.makedirs(bdir, exist_ok=True)
    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=min(len(srcs) + 1, os.cpu_count() or 4)) as ex:
        pending = ex.submit(build_module) if module else None
        results = list(ex.map(lambda src: _compile(src, debug), srcs))
    with open(os.path.join(bdir, "ptxas.log"), "w") as f:
        for (obj, log), src in zip(results, srcs):
            f.write(f"==== {os.path.basename(src)}\n{log}\n")
    tmp = lib + ".tmp"
    cmd = [nvcc(), *ARCH, "-shared", "-cudart", "static", "-o", tmp,
           *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if pending:
        pending.result()
    if verbose:
        print(f"built {lib}", file=sys.stderr)
    return lib


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, debug="--debug" in sys.argv)
