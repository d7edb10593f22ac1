"""Builds libmoba.so in-tree from csrc/*.cu for sm_100a (nvcc cross-compiles without a GPU), and
its MOBA_CHECKS variant libmoba_checks.so (every device-side index derived from data on the device
checked against its buffer; see csrc/common.cuh), and the binding's argument marshalling _bind.so
(csrc/bind.cpp, against the installed torch's headers; the library works without it).

    python -m block_sparse_long_moba_b200.build [--force] [--verbose] [--checks]
"""
from __future__ import annotations

import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmoba.so")
LIB_CHECKS = os.path.join(HERE, "libmoba_checks.so")
BIND = os.path.join(HERE, "_bind.so")
BIND_SRC = os.path.join(CSRC, "bind.cpp")
OBJ_DIR = os.path.join(HERE, "_build")
BIND_STAMP = os.path.join(OBJ_DIR, "bind_made_for.txt")
OBJ_DIR_CHECKS = os.path.join(HERE, "_build_checks")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-Xptxas", "-O3"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the MoBA CUDA library cannot be built")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(
        os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.h")))


def needs_build(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return True
    t = os.path.getmtime(lib)
    return any(os.path.getmtime(p) > t for p in _deps())


def _bind_made_for() -> str:
    """What a _bind.so is tied to beside its sources."""
    import torch
    return f"torch {torch.__version__}, python {sys.version_info[0]}.{sys.version_info[1]}"


def bind_needs_build() -> bool:
    deps = [BIND_SRC, os.path.join(INCLUDE, "moba.h")]
    if not os.path.exists(BIND) or not os.path.exists(BIND_STAMP):
        return True
    if any(os.path.getmtime(p) > os.path.getmtime(BIND) for p in deps):
        return True
    with open(BIND_STAMP) as f:
        return f.read() != _bind_made_for()


def build_bind(force: bool = False):
    """Compile csrc/bind.cpp to _bind.so and return its path, or None where there is no torch with
    CUDA to build it against (libmoba.so does not need it)."""
    try:
        import torch
    except ImportError:
        return None
    if torch.version.cuda is None:
        return None
    if not force and not bind_needs_build():
        return BIND
    import sysconfig

    from torch.utils import cpp_extension
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    inc = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], cuda]
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = BIND + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           f'-DMOBA_TORCH_VERSION="{torch.__version__}"',
           *(f"-isystem{p}" for p in inc), BIND_SRC, "-o", tmp, f"-L{libs}", f"-Wl,-rpath,{libs}",
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("g++ failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, BIND)
    os.makedirs(OBJ_DIR, exist_ok=True)
    with open(BIND_STAMP, "w") as f:
        f.write(_bind_made_for())
    return BIND


def build(force: bool = False, verbose: bool = False, extra_flags=(), checks: bool = False) -> str:
    """Compile every csrc/*.cu to an object and link libmoba.so (libmoba_checks.so with
    checks=True, compiled with -DMOBA_CHECKS=1), and _bind.so where torch has CUDA. Returns the
    library path."""
    lib = _build_library(force, verbose, extra_flags, checks)
    build_bind(force)
    return lib


def _build_library(force, verbose, extra_flags, checks) -> str:
    lib = LIB_CHECKS if checks else LIB
    obj_dir = OBJ_DIR_CHECKS if checks else OBJ_DIR
    flags = [*extra_flags, "-DMOBA_CHECKS=1"] if checks else list(extra_flags)
    if not force and not needs_build(lib):
        return lib
    os.makedirs(obj_dir, exist_ok=True)
    cc = nvcc()
    objs = []
    procs = []
    for src in _sources():
        obj = os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *flags, "-I", INCLUDE, "-c", src, "-o", obj]
        if verbose:
            cmd += ["-Xptxas", "-v"]
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose and text.strip():
            print(text, flush=True)
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    tmp = lib + ".tmp"
    link = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv,
                checks="--checks" in sys.argv))
