"""Compile the CUDA library (kernels + C ABI) for sm_103a, in-tree.

The output is ``host_offload_serving_gb300/_build/libhisparse.so``; it is
rebuilt when a source under ``csrc/`` or ``include/hisparse.h`` is newer.  The
translation units are compiled side by side and linked.
"""
import glob
import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
SRCS = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
HDRS = [os.path.join(ROOT, "include", "hisparse.h"), *sorted(glob.glob(os.path.join(CSRC, "*.cuh")))]
OUT = os.path.join(PKG, "_build", "libhisparse.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc():
    exe = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(exe):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libhisparse")
    return exe


def up_to_date():
    if not os.path.exists(OUT):
        return False
    t = os.path.getmtime(OUT)
    return all(os.path.getmtime(p) <= t for p in (*SRCS, *HDRS, __file__))


def build(force=False, verbose=False):
    if not force and up_to_date():
        return OUT
    os.makedirs(os.path.dirname(OUT), exist_ok=True)
    exe = nvcc()
    tag = f".{os.getpid()}.tmp"
    flags = [*ARCH, "-lineinfo", "-O3", "-std=c++17", "-Xcompiler", "-fPIC",
             "-I", os.path.join(ROOT, "include")]
    if verbose:
        flags.insert(0, "-Xptxas=-v")

    objs = [os.path.join(os.path.dirname(OUT), os.path.basename(src) + tag + ".o") for src in SRCS]

    def compile_one(src, obj):
        cmd = [exe, *flags, "-c", "-o", obj, src]
        if verbose:
            print(" ".join(cmd))
        subprocess.check_call(cmd)

    try:
        with ThreadPoolExecutor(len(SRCS)) as ex:
            list(ex.map(compile_one, SRCS, objs))
        subprocess.check_call([exe, *ARCH, "-shared", "-o", OUT + tag, *objs])
        os.replace(OUT + tag, OUT)
    finally:
        for path in (*objs, OUT + tag):
            if os.path.exists(path):
                os.remove(path)
    return OUT
