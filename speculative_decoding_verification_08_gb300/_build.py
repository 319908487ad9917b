"""Builds libspecverify.so in-tree with nvcc for sm_103a, and the extension that
hands torch tensors to it."""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
CSRC = os.path.join(PKG, "csrc")
SOURCES = [os.path.join(CSRC, "specverify.cu"), os.path.join(CSRC, "cache.cu"),
           os.path.join(CSRC, "cache8.cu"), os.path.join(CSRC, "warp.cu")]
DEPENDS = SOURCES + [os.path.join(CSRC, "sv_device.cuh"), os.path.join(CSRC, "sv_tma.cuh"),
                     os.path.join(CSRC, "sv_item.cuh"), os.path.join(CSRC, "sv_alpha.cuh"),
                     os.path.join(CSRC, "sv_logits.cuh"), os.path.join(CSRC, "sv_debug.cuh"),
                     os.path.join(CSRC, "sv_trace.cuh"), os.path.join(CSRC, "sv_host.cuh"),
                     os.path.join(CSRC, "sv_cache.cuh"), os.path.join(CSRC, "sv_append.cuh"),
                     os.path.join(CSRC, "sv_append8.cuh"), os.path.join(CSRC, "sv_attend8.cuh"),
                     os.path.join(CSRC, "sv_cache_host.cuh"),
                     os.path.join(CSRC, "sv_pairs.cuh"),
                     os.path.join(CSRC, "sv_attend.cuh"), os.path.join(CSRC, "sv_warp.cuh"),
                     os.path.join(CSRC, "sv_tc.cuh"), os.path.join(CSRC, "sv_barrier.cuh"),
                     os.path.join(INCLUDE, "specverify.h")]
LIBRARY = os.path.join(PKG, "libspecverify.so")
# (made for one torch version: the name tells which)
EXTENSION_SOURCE = os.path.join(CSRC, "tensors.cpp")
EXTENSION = os.path.join(PKG, f"_tensors-{importlib.metadata.version('torch')}.so")

NVCC_FLAGS = [
    "-gencode", "arch=compute_103a,code=sm_103a",
    "-lineinfo", "-O3", "-std=c++17",
    "-Xcompiler", "-fPIC", "-shared",
    "-t", "0",   # the sources compile side by side
]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def up_to_date(target: str = LIBRARY, depends=DEPENDS) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in depends)


def extension_command(out: str):
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    include = os.path.join(torch, "include")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            "-I", INCLUDE, "-isystem", include,
            "-isystem", os.path.join(include, "torch", "csrc", "api", "include"),
            "-isystem", sysconfig.get_paths()["include"], EXTENSION_SOURCE, "-o", out,
            "-L", os.path.join(torch, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles the CUDA library and the extension (some seconds each, side by
    side) unless they are up to date."""
    jobs = []
    for target, depends in ((EXTENSION, [EXTENSION_SOURCE, os.path.join(INCLUDE, "specverify.h")]),
                            (LIBRARY, DEPENDS)):
        if not force and up_to_date(target, depends):
            continue
        tmp = target + f".tmp{os.getpid()}"
        if target == LIBRARY:
            cmd = [nvcc(), *NVCC_FLAGS, "-I", INCLUDE, "-o", tmp, *SOURCES]
            if verbose:
                cmd.insert(1, "-Xptxas=-v")
        else:
            cmd = extension_command(tmp)
        jobs.append((subprocess.Popen(cmd), cmd, tmp, target))
    failed = None
    for job, cmd, tmp, target in jobs:
        if job.wait():
            failed = subprocess.CalledProcessError(job.returncode, cmd)
        else:
            os.replace(tmp, target)
    if failed:
        raise failed
    return LIBRARY


def build_variant(out: str, defines) -> str:
    """Compiles the library with extra -D flags into `out`; the regular
    build is left as it is."""
    tmp = out + f".tmp{os.getpid()}"
    cmd = [nvcc(), *NVCC_FLAGS, *defines, "-I", INCLUDE, "-o", tmp, *SOURCES]
    subprocess.run(cmd, check=True)
    os.replace(tmp, out)
    return out


def build_debug(out: str) -> str:
    """A debug build (SV_DEBUG=1): every call checks its input rows for
    negative, NaN or infinite values before its kernels and reports them as
    SV_STATUS_BAD_VALUE."""
    return build_variant(out, ["-DSV_DEBUG=1"])


def build_trace(out: str) -> str:
    """A trace build (SV_TRACE=1): the item kernel records a timeline that
    sv_trace_read returns."""
    return build_variant(out, ["-DSV_TRACE=1"])
