"""Build the CUDA library ``libq4.so`` in-tree with nvcc for sm_100a.

Usage:  python -m post_weight_quantization_group_b200.build [--verbose-ptxas]
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libq4.so")
SOURCES = [os.path.join(CSRC, "q4_api.cu"), os.path.join(CSRC, "kv_api.cu")]
DEPS = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "q4.h")]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libq4.so")


def flags(verbose_ptxas: bool = False) -> list[str]:
    f = [
        "-O3", "-std=c++17", "-lineinfo",
        "-gencode", "arch=compute_100a,code=sm_100a",
        "-Xcompiler", "-fPIC,-fvisibility=hidden",
        "--expt-relaxed-constexpr",
        "-I", INCLUDE, "-I", CSRC,
        "-cudart", "static",
    ]
    if verbose_ptxas:
        f += ["-Xptxas", "-v"]
    return f


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(d) <= t for d in DEPS if os.path.exists(d))


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    base = [nvcc_path(), *flags(verbose_ptxas)]
    with tempfile.TemporaryDirectory() as objs:
        outs = [os.path.join(objs, os.path.basename(src) + ".o") for src in SOURCES]
        jobs = [subprocess.Popen([*base, "-c", src, "-o", o]) for src, o in zip(SOURCES, outs)]
        codes = [j.wait() for j in jobs]
        for src, rc in zip(SOURCES, codes):
            if rc:
                raise subprocess.CalledProcessError(rc, f"nvcc -c {src}")
        fd, tmp = tempfile.mkstemp(suffix=".so", dir=PKG)
        os.close(fd)
        try:
            subprocess.run([*base, "-shared", *outs, "-o", tmp, "-ldl", "-lpthread", "-lrt"], check=True)
            os.replace(tmp, LIB)
        finally:
            if os.path.exists(tmp):
                os.remove(tmp)
    return LIB


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose-ptxas", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force or a.verbose_ptxas, verbose_ptxas=a.verbose_ptxas))
    sys.exit(0)
