"""Builds libdsa.so in-tree with nvcc for sm_103a (GB300), and the Python
binding's extension module _marshal with the host compiler.

Each CUDA translation unit under csrc/ is compiled in parallel to an object
in _build/, then linked (static CUDA runtime) into libdsa.so next to this
file.  Rebuilds only when a source or header is newer than the library (the
extension module also when torch has changed).  The library does not need the
extension module: where that cannot be built (no Python headers, another torch, no
host compiler for it), a warning says why.
"""
from __future__ import annotations

import concurrent.futures
import contextlib
import glob
import os
import shutil
import subprocess
import sysconfig
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libdsa.so")
# measurement variant: the persistent indexer records one globaltimer trace
# record per work item (DSA_ITEM_TRACE) and the tcgen05 forward sums each warp
# role's cycles per pipeline segment (DSA_FWD_PROFILE); nothing else differs
BUILD_TRACE = os.path.join(HERE, "_build_trace")
LIB_TRACE = os.path.join(HERE, "libdsa_trace.so")
# the same item stamps without the indexer's SM-cycle counters, whose clock
# reads in the fold loop make the trace build spill more and run slower: its
# per-item times are the default build's
BUILD_STAMPS = os.path.join(HERE, "_build_stamps")
LIB_STAMPS = os.path.join(HERE, "libdsa_stamps.so")
# checking variant: range checks on gathered rows and shared-memory offsets
# that record a device status (DSA_ERR_INTERNAL) instead of trapping
# (DSA_DEBUG); the arithmetic and results are the default build's
BUILD_DEBUG = os.path.join(HERE, "_build_debug")
LIB_DEBUG = os.path.join(HERE, "libdsa_debug.so")
# the binding's short way into the library (csrc/marshal.cpp), for the Python that its name says and the torch it was
# built with
EXT_SUFFIX = sysconfig.get_config_var("EXT_SUFFIX")
MARSHAL = os.path.join(HERE, "_marshal" + EXT_SUFFIX)
MARSHAL_SOURCE = os.path.join(CSRC, "marshal.cpp")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
              "--expt-relaxed-constexpr", "-I", INCLUDE] + ARCH


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(lib: str) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    deps = sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]
    return any(os.path.getmtime(d) > t for d in deps)


def build_marshal(force: bool = False) -> str:
    """Compile the binding's extension module; returns its path, or raises."""
    import torch
    stamp = os.path.join(BUILD, f"marshal{EXT_SUFFIX}.torch")
    deps = [MARSHAL_SOURCE, os.path.abspath(__file__)] + glob.glob(os.path.join(INCLUDE, "*.h"))
    if not force and os.path.exists(MARSHAL) and os.path.exists(stamp):
        with open(stamp) as f:
            same = f.read() == torch.__version__
        if same and all(os.path.getmtime(d) <= os.path.getmtime(MARSHAL) for d in deps):
            return MARSHAL
    os.makedirs(BUILD, exist_ok=True)
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           f'-DDSA_TORCH_VERSION="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", os.path.join(root, "include"),
           "-I", os.path.join(root, "include", "torch", "csrc", "api", "include"), "-I", os.path.join(cuda, "include"),
           "-I", sysconfig.get_paths()["include"], MARSHAL_SOURCE, "-o", tmp, "-L", os.path.join(root, "lib"),
           *[f"-l{n}" for n in ("c10", "c10_cuda", "torch_cpu", "torch_cuda", "torch", "torch_python")]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"marshal.cpp failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, MARSHAL)
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return MARSHAL


def _try_marshal(force: bool):
    """Build the extension module; returns why it could not be built (the Python code then does every call), or None."""
    plain = os.path.join(os.path.dirname(MARSHAL), "_marshal.so")  # a name that any Python would import
    if plain != MARSHAL:
        _remove(plain)
    try:
        build_marshal(force)
    except Exception as e:
        _remove(MARSHAL)  # made of other sources, or for another torch
        return e
    return None


def _remove(path: str) -> None:
    with contextlib.suppress(FileNotFoundError):  # (another process may build, too)
        os.remove(path)


def _warn_marshal(why) -> None:
    if why is not None:
        warnings.warn(f"the extension module was not built, calls will take more of the host's time: {why}", RuntimeWarning,
                      stacklevel=3)


def build(force: bool = False, verbose: bool = False, trace: bool = False, debug: bool = False,
          stamps: bool = False) -> str:
    """Compile and link libdsa.so (or, with trace=True, the measurement
    variant libdsa_trace.so, with stamps=True its stamps-only form
    libdsa_stamps.so, or with debug=True the range-checking variant
    libdsa_debug.so); returns its path."""
    if trace + debug + stamps > 1:
        raise ValueError("build: the trace, stamps and debug variants are separate builds")
    default = not (trace or stamps or debug)
    lib, bdir = (LIB_TRACE, BUILD_TRACE) if trace else (LIB_STAMPS, BUILD_STAMPS) if stamps else \
        (LIB_DEBUG, BUILD_DEBUG) if debug else (LIB, BUILD)
    if not force and not _stale(lib):
        if default:
            _warn_marshal(_try_marshal(False))
        return lib
    os.makedirs(bdir, exist_ok=True)
    nvcc = _nvcc()
    flags = NVCC_FLAGS + (["-DDSA_ITEM_TRACE=1", "-DDSA_FWD_PROFILE=1"] if trace or stamps else []) + \
        (["-DDSA_TRACE_STAMPS_ONLY=1"] if stamps else []) + (["-DDSA_DEBUG=1"] if debug else [])

    def compile_one(src: str) -> str:
        obj = os.path.join(bdir, os.path.basename(src)[:-3] + ".o")
        cmd = [nvcc, *flags, "-c", src, "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        if verbose and r.stderr:
            print(r.stderr)
        return obj

    srcs = sources()
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(srcs) + 1) as ex:
        marshal = ex.submit(_try_marshal, force) if default else None
        objs = list(ex.map(compile_one, srcs))
    tmp = lib + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    if marshal is not None:
        _warn_marshal(marshal.result())
    return lib


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
