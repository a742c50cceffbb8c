"""Build libmoe.so (the CUDA path) in-tree with nvcc for sm_103a, and the
Python module that calls its small operators (csrc/fastcall.c; left out where
Python has no headers).

Each translation unit under csrc/ compiles to an object in parallel; the
objects link into sparse_moe_expert_02_gb300/_build/libmoe.so with the CUDA
runtime linked statically.  Nothing here runs on the GPU.
"""
from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmoe.so")
FAST = os.path.join(BUILD, "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe")


def python_headers():
    """The folder of Python.h, or None: libmoe does without, only the small operators' module needs it."""
    inc = sysconfig.get_paths()["include"]
    return inc if os.path.exists(os.path.join(inc, "Python.h")) else None


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _fingerprint(flags) -> str:
    h = hashlib.sha256()
    for f in sorted(_sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.c"))
                    + glob.glob(os.path.join(INCLUDE, "*.h"))):
        h.update(f.encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(flags).encode())
    return h.hexdigest()


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile (if sources changed) and return the path of libmoe.so."""
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-fvisibility=hidden",
                    "--expt-relaxed-constexpr", "-I", INCLUDE, "-I", CSRC] + list(extra_flags)
    fp = _fingerprint(flags)
    stamp = os.path.join(BUILD, "libmoe.stamp")
    headers = python_headers()
    if not force and os.path.exists(LIB) and (os.path.exists(FAST) or not headers) and os.path.exists(stamp) and open(stamp).read() == fp:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()

    def one(src):
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        cmd = [cc] + flags + ["-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    def fast():
        if not headers:
            if os.path.exists(FAST):
                os.remove(FAST)  # of other sources
            return
        tmp = FAST + f".tmp{os.getpid()}"
        r = subprocess.run([cc, "-O2", "-shared", "-cudart", "none", "-Xcompiler", "-fPIC,-fvisibility=hidden", "-I", INCLUDE, "-I",
                            headers, os.path.join(CSRC, "fastcall.c"), "-o", tmp], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"fastcall.c failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, FAST)

    srcs = _sources()
    with ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        small = ex.submit(fast)
        objs = list(ex.map(one, srcs))
        small.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp, "w") as fh:
        fh.write(fp)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
