"""Build libwb.so in-tree with nvcc for sm_103a (no cmake, no torch extension).

Each CUDA translation unit is compiled in parallel, then linked into
``whisper_encoder_gb300/_build/libwb.so`` (git-ignored); ``--debug`` builds the
bounds-checked variant into ``_build_debug/libwb_debug.so``.  ``wb_host.so``, the C++
marshalling of a few calls, is built beside it with g++ against the installed torch; it only
saves host time, so a machine that cannot build it goes without.  Usage:
    python -m whisper_encoder_gb300.build [--force] [--verbose-ptxas] [--debug]
"""
from __future__ import annotations

import concurrent.futures as cf
import hashlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libwb.so")
LIB_HOST = os.path.join(BUILD, "wb_host.so")
BUILD_DEBUG = os.path.join(HERE, "_build_debug")
LIB_DEBUG = os.path.join(BUILD_DEBUG, "libwb_debug.so")
SOURCES = ["api.cu", "kernels.cu", "tc_kernels.cu", "static_scratch.cu", "host_pipeline.cu", "layernorm_train.cu", "head_loss.cu",
           "cross_attention.cu", "grad_clip.cu", "policy_loss.cu"]
HOST_SOURCE = "host_calls.cpp"
HOST_FLAGS = ["-O2", "-std=c++17", "-fPIC", "-shared"]
ARCH = "-gencode=arch=compute_103a,code=sm_103a"


def _nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found")


def _flags(ptxas_verbose: bool = False, debug: bool = False):
    f = [ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-I" + os.path.join(ROOT, "include")]
    if debug:
        f.append("-DWB_DEBUG=1")
    if ptxas_verbose:
        f.append("-Xptxas=-v")
    return f


def _digest(debug: bool = False) -> str:
    h = hashlib.sha256()
    for name in sorted(os.listdir(CSRC)):
        if name == HOST_SOURCE:
            continue
        with open(os.path.join(CSRC, name), "rb") as fh:
            h.update(name.encode() + fh.read())
    with open(os.path.join(ROOT, "include", "wb.h"), "rb") as fh:
        h.update(fh.read())
    h.update(" ".join(_flags(debug=debug)).encode())
    return h.hexdigest()


def _host_command(out: str) -> list:
    torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)
    nvcc = os.path.realpath(_nvcc())
    include = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include")]
    libs = os.path.join(torch_dir, "lib")
    return [os.environ.get("CXX", "g++"), *HOST_FLAGS, *["-I" + d for d in include], os.path.join(CSRC, HOST_SOURCE),
            "-o", out, "-L" + libs, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath," + libs]


def _host_digest() -> str:
    """What wb_host.so depends on: its source, wb.h, the torch and Python it is for.  Not where the compilers lie: a machine without them runs
    a tree that was built."""
    h = hashlib.sha256("\n".join((importlib.metadata.version("torch"), sys.version, sysconfig.get_platform(), *HOST_FLAGS)).encode())
    for path in (os.path.join(CSRC, HOST_SOURCE), os.path.join(ROOT, "include", "wb.h")):
        with open(path, "rb") as fh:
            h.update(fh.read())
    return h.hexdigest()


def build_host(force: bool = False) -> str | None:
    """Compile wb_host.so against the installed torch (if its source, wb.h or torch changed); None where that fails."""
    stamp = os.path.join(BUILD, "host_digest.txt")
    stale = False
    try:
        digest, current = _host_digest(), False
        if os.path.exists(LIB_HOST) and os.path.exists(stamp):
            with open(stamp) as fh:
                current = fh.read() == digest
        stale = not current
        if current and not force:
            return LIB_HOST
        cmd = _host_command(LIB_HOST + ".tmp")
        os.makedirs(BUILD, exist_ok=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(r.stderr[-2000:])
        os.replace(LIB_HOST + ".tmp", LIB_HOST)
        with open(stamp, "w") as fh:
            fh.write(digest)
        return LIB_HOST
    except Exception as e:  # noqa: BLE001 - the package works without it, with more host time a call
        if stale and os.path.exists(LIB_HOST):
            os.remove(LIB_HOST)          # of another torch or another wb.h
        sys.stderr.write(f"wb_host.so is not built: {e}\n")
        return None


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = True, debug: bool = False) -> str:
    """Compile (if sources changed) and return the path of libwb.so.

    debug=True builds the bounds-checked variant (-DWB_DEBUG) as _build_debug/libwb_debug.so."""
    out_dir = BUILD_DEBUG if debug else BUILD
    lib_path = LIB_DEBUG if debug else LIB
    os.makedirs(out_dir, exist_ok=True)
    stamp = os.path.join(out_dir, "digest.txt")
    dg = _digest(debug)
    if not force and os.path.exists(lib_path) and os.path.exists(stamp) and open(stamp).read() == dg:
        if not debug:
            build_host()
        return lib_path
    nvcc = _nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(out_dir, src.replace(".cu", ".o"))
        cmd = [nvcc, *_flags(ptxas_verbose, debug), "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        host = None if debug else ex.submit(build_host, force)
        for obj, log in ex.map(compile_one, SOURCES):
            objs.append(obj)
            if log and (ptxas_verbose or not quiet):
                sys.stderr.write(log)
        if host:
            host.result()
    tmp = lib_path + ".tmp"
    cmd = [nvcc, ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib_path)
    with open(stamp, "w") as fh:
        fh.write(dg)
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, ptxas_verbose="--verbose-ptxas" in sys.argv, quiet=False,
                debug="--debug" in sys.argv))
