"""Builds libmoe_gb300.so in-tree with nvcc for sm_103a.

Each .cu translation unit is compiled in parallel, then linked into one
shared library that exports the C ABI of include/moe_gb300.h.  The CUDA
runtime is linked statically; the driver (libcuda) is reached through
cudaGetDriverEntryPointByVersion, so loading the library needs no GPU.
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libmoe_gb300.so")
FAST = os.path.join(HERE, "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX"))
SOURCES = ["abi.cu", "router.cu", "route_dispatch.cu", "dispatch.cu", "dispatch_static.cu", "ffn.cu",
           "ffn_decode.cu", "macs.cu", "calib.cu", "cast.cu", "qk_rope.cu", "attn_kv4.cu", "attn_kv4_prefill.cu", "kv4_pages.cu"]
HEADERS = ["common.cuh", "launch.h", "routing.cuh", "permute.cuh", "kv4.cuh", "attn_kv4.cuh", "ranges.h", "tmap.h", "../../include/moe_gb300.h"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _newest_input() -> float:
    paths = [os.path.join(CSRC, f) for f in SOURCES + HEADERS]
    paths.append(os.path.join(os.path.dirname(HERE), "include", "moe_gb300.h"))
    paths.append(os.path.join(CSRC, "fastcall.c"))
    paths.append(os.path.abspath(__file__))
    return max(os.path.getmtime(p) for p in paths)


def _build_fastcall() -> None:
    """The CPython module that calls the attention operators without ctypes."""
    cc = os.environ.get("CC") or shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        raise RuntimeError("no C compiler found")
    tmp = FAST + ".tmp%d" % os.getpid()
    cmd = [cc, "-shared", "-fPIC", "-O2", "-Wall", "-I", sysconfig.get_paths()["include"], os.path.join(CSRC, "fastcall.c"), "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("building fastcall.c failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, FAST)


def build(force: bool = False, verbose: bool = False) -> str:
    built = all(os.path.exists(p) and os.path.getmtime(p) >= _newest_input() for p in (LIB, FAST))
    if not force and built:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v" if verbose else "-O3",
                    "--expt-relaxed-constexpr", "-I", CSRC]

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [cc, "-c", os.path.join(CSRC, src), "-o", obj] + flags
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, r.stdout, r.stderr))
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        fast = ex.submit(_build_fastcall)
        objs = list(ex.map(compile_one, SOURCES))
        fast.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [cc, "-shared", "-o", tmp] + objs + ARCH + ["-cudart", "static", "-Xcompiler", "-fPIC"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
