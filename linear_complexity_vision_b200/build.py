"""Build libvrwkv.so (the sm_100a CUDA library behind include/vrwkv.h) in-tree."""
from __future__ import annotations

import os
import re
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libvrwkv.so")
SOURCES = ["vrwkv_api.cu", "decay_attn_api.cu", "layer_norm_api.cu"]
OBJ = os.path.join(PKG, "build")  # object files, one per source

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-lineinfo", "-O3",
              "-std=c++17", "-Xcompiler", "-fPIC,-O2",
              "-I" + os.path.join(ROOT, "include"), "-I" + CSRC]
LIBS: list = []


def _deps(source: str, seen=None) -> set:
    """A source file and the project headers it includes, by path."""
    seen = set() if seen is None else seen
    for base in (CSRC, os.path.join(ROOT, "include")):
        path = os.path.join(base, source)
        if os.path.exists(path) and path not in seen:
            seen.add(path)
            with open(path) as f:
                for name in re.findall(r'^\s*#include "([^"]+)"', f.read(), flags=re.M):
                    _deps(name, seen)
    return seen


def _object(source: str) -> str:
    return os.path.join(OBJ, os.path.splitext(source)[0] + ".o")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the sources that are newer than the library (one object file
    each, in parallel) and link them."""
    deps = {s: _deps(s) for s in SOURCES}
    if not force and not _stale(LIB, set().union(*deps.values())):
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    os.makedirs(OBJ, exist_ok=True)
    flags = NVCC_FLAGS + (["-Xptxas=-v"] if verbose else [])
    running = []
    for s in SOURCES:
        if force or _stale(_object(s), deps[s]):
            tmp = _object(s) + f".tmp{os.getpid()}"
            cmd = [nvcc, *flags, "-c", "-o", tmp, os.path.join(CSRC, s)]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            running.append((cmd, tmp, _object(s), subprocess.Popen(cmd)))
    for cmd, tmp, obj, proc in running:
        if proc.wait() != 0:
            for _, _, _, other in running:
                other.wait()
            raise subprocess.CalledProcessError(proc.returncode, cmd)
        os.replace(tmp, obj)
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([nvcc, *NVCC_FLAGS, "-shared", "-o", tmp, *[_object(s) for s in SOURCES], *LIBS], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
