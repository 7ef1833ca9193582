"""Build libsffn.so (the C-ABI library) in-tree for sm_100a with nvcc.

    python -m activation_sparse_gated_relu_b200.build [--force]
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
LIB = os.path.join(HERE, "libsffn.so")
HEADER = os.path.join(ROOT, "include", "sffn.h")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC"]
UNITS = ["sffn.cu", "layer.cu"]   # translation units, compiled side by side


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsffn.so")


def _sources() -> list[str]:
    files = [HEADER]
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh", ".h")):
            files.append(os.path.join(CSRC, f))
    return files


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(f) <= t for f in _sources())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/ into libsffn.so next to this file; return its path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    with tempfile.TemporaryDirectory() as tmp_dir:
        objects, running = [], []
        for unit in UNITS:
            obj = os.path.join(tmp_dir, unit + ".o")
            cmd = [nvcc, *NVCC_FLAGS, "-c", "-o", obj, os.path.join(CSRC, unit)]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            log = open(obj + ".log", "w+")
            running.append((subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT), log))
            objects.append(obj)
        failed = []
        for proc, log in running:
            if proc.wait() != 0:
                log.seek(0)
                failed.append(log.read())
            log.close()
        if failed:
            raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
        tmp = LIB + ".tmp"
        cmd = [nvcc, *ARCH, "-Xcompiler", "-fPIC", "-shared", "-o", tmp, *objects]
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed:\n" + res.stdout + res.stderr)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
