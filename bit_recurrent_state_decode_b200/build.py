"""Build libqstate.so and libqmixer.so in-tree with nvcc for sm_100a.

    python -m bit_recurrent_state_decode_b200.build [--force] [-v]

libqstate.so (csrc/) is the quantized recurrent-state step, libqmixer.so
(csrc/mixer/) the operators around it, and _qmixer_usual.so (csrc/mixer/binding/) the
module that makes their usual calls from Python.  Each .cu unit is compiled in parallel,
then each library is linked with a static CUDA runtime; a library whose
sources are older than it is left alone.  The two libraries need nvcc alone; the
module needs PyTorch's headers and g++ too and is left out, with a message, where no
PyTorch with CUDA is installed.  It is built for one version of PyTorch and of Python, whose
numbers it holds: another one builds it anew.  No fast-math: the step's arithmetic
is specified to the bit (see include/qstate.h), so FMA contraction is disabled
and every fused multiply-add in the kernels is written explicitly.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libqstate.so")
MIXER_LIB = os.path.join(PKG, "libqmixer.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
CFLAGS = ARCH + ["-O3", "-std=c++17", "-lineinfo", "-fmad=false", "-Xcompiler", "-fPIC",
                 "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]


# library -> folder of its units, public headers
LIBS = {LIB: (CSRC, ("qstate.h",)), MIXER_LIB: (os.path.join(CSRC, "mixer"), ("qstate.h", "qmixer.h"))}

USUAL = os.path.join(PKG, "_qmixer_usual.so")
USUAL_SRC = os.path.join(CSRC, "mixer", "binding", "qmixer_usual.cpp")


def _deps(lib):
    src, headers = LIBS[lib]
    return ([f for ext in ("*.cu", "*.cuh", "*.h") for f in glob.glob(os.path.join(src, ext))]
            + [os.path.join(ROOT, "include", h) for h in headers] + [__file__])


def _lib_up_to_date(lib) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps(lib))


def usual_versions() -> str:
    """What the module's binary interface goes by: the interpreter's and PyTorch's versions
    ("" without a PyTorch that uses CUDA)."""
    try:
        import torch
    except ImportError:
        return ""
    return "" if torch.version.cuda is None else f"{sys.implementation.cache_tag} torch {torch.__version__}"


def usual_built_for(versions: str) -> bool:
    """Whether the module in the package was built for these versions."""
    try:
        with open(USUAL, "rb") as f:
            return f"[built for {versions}]".encode() in f.read()
    except FileNotFoundError:
        return False


def _usual_up_to_date() -> bool:
    versions = usual_versions()
    if not versions:                 # nothing could load it
        return True
    return usual_built_for(versions) and all(
        os.path.getmtime(d) <= os.path.getmtime(USUAL)
        for d in (USUAL_SRC, os.path.join(ROOT, "include", "qmixer.h"), __file__))


def up_to_date() -> bool:
    return all(_lib_up_to_date(lib) for lib in LIBS) and _usual_up_to_date()


def _build_usual():
    import sysconfig

    versions = usual_versions()
    if not versions:
        print("no PyTorch with CUDA is installed: _qmixer_usual.so, which qmixer.py uses, is left out", file=sys.stderr)
        return
    from torch.utils import cpp_extension
    tmp = USUAL + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-o", tmp, USUAL_SRC,
           f'-DBUILT_FOR="[built for {versions}]"', "-I" + os.path.join(ROOT, "include"), "-I" + sysconfig.get_paths()["include"],
           "-I/usr/local/cuda/include"]
    cmd += ["-isystem" + d for d in cpp_extension.include_paths()]
    cmd += [f for d in cpp_extension.library_paths() for f in ("-L" + d, "-Wl,-rpath," + d)]
    cmd += ["-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python", "-L" + PKG, "-lqmixer", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"the compiler failed on {USUAL_SRC}:\n{r.stderr}")
    os.replace(tmp, USUAL)


def build(force: bool = False, verbose: bool = False) -> str:
    stale = [lib for lib in LIBS if force or not _lib_up_to_date(lib)]
    if not stale:
        if force or not _usual_up_to_date():
            _build_usual()
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [NVCC] + CFLAGS + extra + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stderr}")
        return obj, r.stderr

    with concurrent.futures.ThreadPoolExecutor(max_workers=os.cpu_count() or 4) as ex:
        units = {lib: sorted(glob.glob(os.path.join(LIBS[lib][0], "*.cu"))) for lib in stale}
        results = {lib: [ex.submit(compile_one, src) for src in srcs] for lib, srcs in units.items()}
        for lib in stale:
            done = [r.result() for r in results[lib]]
            if verbose:
                for _, err in done:
                    sys.stderr.write(err)
            tmp = lib + ".tmp"
            cmd = [NVCC] + ARCH + ["-shared", "-cudart", "static", "-o", tmp] + [o for o, _ in done]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"link failed:\n{r.stderr}")
            os.replace(tmp, lib)
    _build_usual()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
