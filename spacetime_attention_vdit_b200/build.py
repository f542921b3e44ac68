"""Build libvdit.so in place (sm_100a) with nvcc.

    python -m spacetime_attention_vdit_b200.build [--verbose-ptxas]

csrc/vdit_api.cu includes every kernel that waits (the watchdog's flag is one
symbol of that translation unit); the block selection, whose kernels have no
waits, is compiled on its own and linked in as an object.  The CUDA runtime is
linked statically and the driver's tensor-map encoder is looked up at run time,
so the .so needs no CUDA libraries on its link line.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libvdit.so")
SOURCES = [os.path.join(CSRC, "vdit_api.cu")]
OBJECT_SOURCES = [os.path.join(CSRC, "block_select.cu")]
DEPS = SOURCES + OBJECT_SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
    os.path.join(INCLUDE, "vdit.h")]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libvdit.so")


FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]


def command(ptxas_verbose: bool = False, out: str = LIB, objects=()):
    """Compile vdit_api.cu and link it with ``objects`` into the shared library."""
    verbose = ["-Xptxas", "-v"] if ptxas_verbose else []
    return [nvcc()] + verbose + FLAGS + ["-shared", "-cudart", "static", "-o", out] + SOURCES + list(objects)


def object_command(source: str, out: str, ptxas_verbose: bool = False):
    """Compile one of OBJECT_SOURCES on its own."""
    verbose = ["-Xptxas", "-v"] if ptxas_verbose else []
    return [nvcc()] + verbose + FLAGS + ["-c", "-o", out, source]


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in DEPS)


def build(force: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile the library unless it is newer than every source; returns its path."""
    if not force and not ptxas_verbose and up_to_date():
        return LIB
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as folder:
        objects = [os.path.join(folder, os.path.basename(src) + ".o") for src in OBJECT_SOURCES]
        steps = [object_command(src, obj, ptxas_verbose) for src, obj in zip(OBJECT_SOURCES, objects)]
        for cmd in steps + [command(ptxas_verbose, tmp, objects)]:
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
            if ptxas_verbose:
                sys.stderr.write(res.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force=True, ptxas_verbose="--verbose-ptxas" in sys.argv)
    print(LIB)
