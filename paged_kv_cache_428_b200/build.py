"""Build libpa.so in-tree: nvcc for sm_100a (device code) + the host C++ sources.

    python paged_kv_cache_428_b200/build.py [--verbose-ptxas]

The .so lands next to this file, where the Python binding loads it from.  This script
imports nothing from the package, so it runs before the library exists.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor
from pathlib import Path

PKG = Path(__file__).resolve().parent
ROOT = PKG.parent
CSRC = PKG / "csrc"
OBJ = PKG / "_build"
LIB = PKG / "libpa.so"
SOURCES = [CSRC / f for f in ("pa_lib.cu", "pa_block_scales.cu", "pa_evict.cu", "pa_scoremod.cu", "pa_prefill_scoremod.cu", "host.cpp", "allocator.cpp")]
HEADERS = [ROOT / "include" / "pa.h"] + sorted(CSRC.glob("*.cuh"))

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC",
    "--expt-relaxed-constexpr",
]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def stale() -> bool:
    if not LIB.exists():
        return True
    t = LIB.stat().st_mtime
    return any(p.stat().st_mtime > t for p in SOURCES + HEADERS)


def _object(src: Path, force: bool, extra: list) -> Path:
    """The object file of one source, compiled if it is older than a file that it was made from."""
    obj, dep = OBJ / (src.name + ".o"), OBJ / (src.name + ".d")
    if not force and obj.exists() and dep.exists():
        names = dep.read_text().replace("\\\n", " ").split(":", 1)[1].split()
        made_from = [Path(n) for n in names if Path(n).is_relative_to(ROOT)]
        if all(p.exists() and p.stat().st_mtime <= obj.stat().st_mtime for p in made_from):
            return obj
    cmd = [nvcc(), *NVCC_FLAGS, *extra, "-I", str(ROOT / "include"), "-I", str(CSRC), "-MD", "-MF", str(dep), "-c", str(src),
           "-o", str(obj)]
    subprocess.run(cmd, check=True)
    return obj


def build(verbose_ptxas: bool = False, force: bool = False) -> Path:
    if not force and not stale():
        return LIB
    OBJ.mkdir(exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []
    with ThreadPoolExecutor(max_workers=len(SOURCES)) as pool:      # one compiler process per source
        objects = list(pool.map(lambda src: _object(src, force, extra), SOURCES))
    subprocess.run([nvcc(), *NVCC_FLAGS, "-shared", *map(str, objects), "-o", str(LIB)], check=True)
    return LIB


if __name__ == "__main__":
    build(verbose_ptxas="--verbose-ptxas" in sys.argv, force=True)
    print(LIB)
