"""Build libspecverify.so (and libspecverify_debug.so, whose verify calls count
failed bounds checks; the cache calls check theirs in both) in-tree with nvcc for sm_100a: one object per translation unit, compiled in
parallel, then one link."""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
HDR = os.path.join(ROOT, "include", "spec_verify.h")
# translation units, each with the files that it includes
UNITS = {
    "library.cu": ["spec_verify.cu", "internal.h"],
    "spec_cache.cu": ["internal.h", "cache_device.cuh"],
    "spec_attention.cu": ["internal.h", "cache_device.cuh"],
}
SRC = sorted({os.path.join(CSRC, f) for unit, inc in UNITS.items() for f in [unit, *inc]})
OBJ = os.path.join(PKG, "_build")
OUT = os.path.join(PKG, "libspecverify.so")
OUT_DEBUG = os.path.join(PKG, "libspecverify_debug.so")

NVCC_ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = [*NVCC_ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC"]
LINK_FLAGS = [*NVCC_ARCH, "-shared", "-cudart", "static"]
DEBUG_FLAGS = ["-DSPEC_DEBUG_BOUNDS"]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _older(out: str, deps) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(p) > t for p in deps)


def stale(out: str = OUT) -> bool:
    return _older(out, SRC + [HDR, __file__])


def _objects(out: str):
    """(object, source, files that it depends on) of each translation unit of a library."""
    kind = "debug" if out == OUT_DEBUG else "release"
    for unit, inc in UNITS.items():
        src = os.path.join(CSRC, unit)
        obj = os.path.join(OBJ, f"{os.path.splitext(unit)[0]}.{kind}.o")
        yield obj, src, [src, HDR, __file__, *(os.path.join(CSRC, f) for f in inc)]


def _run(cmds, verbose):
    procs = []
    for what, cmd in cmds:
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        procs.append((what, subprocess.Popen(cmd)))
    failed = [what for what, p in procs if p.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, f"nvcc ({', '.join(failed)})")


def build(force: bool = False, verbose: bool = False, debug: bool = True) -> str:
    """Compile the library (and, with ``debug``, the bounds-checked one) when a
    source is newer than it; objects that are still current are kept.  Returns the
    path of the library."""
    jobs = [(o, x) for o, x in [(OUT, []), (OUT_DEBUG, DEBUG_FLAGS)] if (o == OUT or debug) and (force or stale(o))]
    os.makedirs(OBJ, exist_ok=True)
    compiles = []
    for out, extra in jobs:
        for obj, src, deps in _objects(out):
            if force or _older(obj, deps):
                compiles.append((obj, [nvcc(), *NVCC_FLAGS, *extra, "-I", os.path.join(ROOT, "include"), "-c", src,
                                       "-o", obj + ".tmp"]))
    _run(compiles, verbose)
    for obj, _ in compiles:
        os.replace(obj + ".tmp", obj)
    _run([(out, [nvcc(), *LINK_FLAGS, *(obj for obj, _, _ in _objects(out)), "-o", out + ".tmp"]) for out, _ in jobs],
         verbose)
    for out, _ in jobs:
        os.replace(out + ".tmp", out)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
