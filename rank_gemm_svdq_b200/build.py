"""Build libsvdq.so in-tree: nvcc for the sm_100a kernels, g++ (OpenMP) for the
host half, linked into one shared library next to this file."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT = os.path.join(HERE, "libsvdq.so")
BUILD = os.path.join(HERE, "_build")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]

SOURCES_CU = ["svdq_device.cu", "kv_device.cu", "paged_device.cu"]
SOURCES_CPP = ["svdq_host.cpp"]
HEADERS = ["internal.h", "layout.h", "ptx.cuh"]


def _stale(target: str, deps: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(HERE, "..", "include", "svdq.h"),
                                                        os.path.abspath(__file__)]
    objs, running = [], []                       # the sources are compiled at the same time
    for src in SOURCES_CU + SOURCES_CPP:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src + ".o")
        objs.append(o)
        if not force and not _stale(o, [s] + hdrs):
            continue
        if src in SOURCES_CU:
            cmd = [NVCC, *ARCH, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
                   "--expt-relaxed-constexpr", "-c", s, "-o", o]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
        else:
            cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fopenmp", "-ffp-contract=off", "-c", s, "-o", o]
        running.append((cmd, o, subprocess.Popen(cmd)))
    failed = [(cmd, o, p.returncode) for cmd, o, p in running if p.wait() != 0]
    for cmd, o, _ in failed:
        if os.path.exists(o):
            os.remove(o)
    if failed:
        raise subprocess.CalledProcessError(failed[0][2], failed[0][0])
    if force or _stale(OUT, objs):
        tmp = OUT + f".{os.getpid()}.tmp"
        subprocess.check_call([NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static",
                               "-Xcompiler", "-fopenmp", "-lgomp"])
        os.replace(tmp, OUT)
    return OUT


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
