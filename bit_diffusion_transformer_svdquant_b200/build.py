"""Builds libsvdq.so (the sm_100a C-ABI library) in-tree with nvcc.

The library links the CUDA runtime statically and reaches the driver only through the runtime's
entry-point query, so it loads (and exports its symbols) on machines without a GPU driver.
"""
from __future__ import annotations

import os
import re
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO, "include")
LIB_PATH = os.path.join(PKG_DIR, "libsvdq.so")
SOURCES = [os.path.join(CSRC, f) for f in ("svdq.cu", "svdq_fp8b.cu", "svdq_heads.cu")]

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-cudart", "static",
]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def includes(path: str) -> set[str]:
    """The file and every header of this repository that it includes, directly or not."""
    found, todo = set(), [path]
    while todo:
        p = todo.pop()
        if p in found:
            continue
        found.add(p)
        with open(p) as f:
            for name in re.findall(r'^\s*#include "([^"]+)"', f.read(), re.M):
                todo += [q for q in (os.path.join(d, name) for d in (CSRC, INCLUDE)) if os.path.exists(q)]
    return found


DEPS = sorted(set().union(*(includes(s) for s in SOURCES)))


def _current(target: str, deps, flags) -> bool:
    """Whether a file is newer than all it was made from and was made with these flags (recorded beside it)."""
    if not os.path.exists(target) or not os.path.exists(target + ".flags"):
        return False
    with open(target + ".flags") as f:
        if f.read() != "\n".join(flags):
            return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(d) <= t for d in deps)


def _make(target: str, flags, cmd, verbose):
    """Runs the command that writes target + ".tmp"; the file is then replaced, with the record of its flags."""
    _run(cmd, verbose)
    if os.path.exists(target + ".flags"):
        os.remove(target + ".flags")
    os.replace(target + ".tmp", target)
    with open(target + ".flags", "w") as f:
        f.write("\n".join(flags))


def up_to_date(extra=None) -> bool:
    return _current(LIB_PATH, DEPS, [*NVCC_FLAGS, *(extra or [])])


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stderr}\n{res.stdout}")
    if verbose and res.stderr:
        print(res.stderr, file=sys.stderr)


def build(force: bool = False, verbose: bool = False, extra=None) -> str:
    """One object per source, compiled side by side (an object that is newer than all its source includes
    and has the same flags is kept), linked into the library."""
    if not force and up_to_date(extra):
        return LIB_PATH
    flags = [*NVCC_FLAGS, *(extra or [])]
    cmd = [nvcc(), *flags, "-I", INCLUDE, "-I", CSRC]

    def compile_one(src):
        obj = src[:-3] + ".o"
        if force or not _current(obj, includes(src), flags):
            _make(obj, flags, [*cmd, "-c", "-o", obj + ".tmp", src], verbose)
        return obj

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        objects = list(pool.map(compile_one, SOURCES))
    _make(LIB_PATH, flags, [*cmd, "-shared", "-o", LIB_PATH + ".tmp", *objects], verbose)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None))
