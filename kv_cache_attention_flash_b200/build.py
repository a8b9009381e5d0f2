"""Builds libfdllm.so (the C-ABI library) in-tree with nvcc for sm_100a, and
_serve.so, the native argument marshalling of the single-token serving calls.

    python -m kv_cache_attention_flash_b200.build [--force] [--verbose]

The library is self-contained: CUDA runtime linked statically, the tensor-map
encoder fetched from the driver at run time, no torch types anywhere. _serve.so
is a Python extension module over torch tensors that calls the library.
"""
from __future__ import annotations

import argparse
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libfdllm.so")
SOURCES = ["api.cu", "step_bf16.cu", "step_f32.cu", "mass_select.cu", "verify.cu", "oproj.cu",
           "serve_api.cu", "blocks.cu", "decode_attn.cu", "linear.cu"]
HEADERS = ["fdllm_internal.h", "host_api.h", "ptx.cuh", "ptx_serve.cuh", "serve_index.h", "serve_internal.h"]

EXT = os.path.join(PKG, "_serve.so")
EXT_SRC = os.path.join(CSRC, "bind.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "--expt-relaxed-constexpr",
    "-Xcompiler", "-fPIC,-O2,-fvisibility=hidden",
    "-Xptxas", "-v",
]


def nvcc_path() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _inputs():
    files = [os.path.join(CSRC, s) for s in SOURCES + HEADERS]
    files.append(os.path.join(INCLUDE, "fdllm.h"))
    files.append(os.path.abspath(__file__))
    return files


def _newer(target: str, inputs) -> bool:
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(f) <= t for f in inputs)


def up_to_date() -> bool:
    return _newer(LIB, _inputs())


def build_ext(force: bool = False) -> str:
    """Builds _serve.so against the installed torch."""
    if not force and _newer(EXT, [EXT_SRC, os.path.join(INCLUDE, "fdllm.h"), os.path.abspath(__file__)]):
        return EXT
    import sysconfig

    import torch
    home = os.path.dirname(os.path.abspath(torch.__file__))
    inc = os.path.join(home, "include")
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc_path())))
    tmp = EXT + ".tmp"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-I", inc, "-I", os.path.join(inc, "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"], EXT_SRC,
           "-o", tmp, "-L", os.path.join(home, "lib"), "-ltorch_python", "-ltorch", "-ltorch_cpu",
           "-ltorch_cuda", "-lc10", "-lc10_cuda"]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout)
        raise RuntimeError("g++ failed for _serve.so")
    os.replace(tmp, EXT)
    return EXT


PROBE_SRC = os.path.join(CSRC, "mma_rate.cu")
PROBE = os.path.join(PKG, "mma_rate")


def build_probe() -> str:
    """Builds the tcgen05.mma issue-rate measurement program (a standalone
    executable beside the library; not used by the library)."""
    subprocess.check_call([nvcc_path(), "-gencode", "arch=compute_100a,code=sm_100a", "-O3",
                           "-std=c++17", "-I", CSRC, "-o", PROBE, PROBE_SRC, "-lcuda"])
    return PROBE


def build(force: bool = False, verbose: bool = False) -> str:
    build_ext(force)
    if not force and up_to_date():
        return LIB
    nvcc = nvcc_path()
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    procs = []
    for s in SOURCES:
        obj = os.path.join(objdir, s.replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", os.path.join(CSRC, s), "-o", obj]
        procs.append((s, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)))
        objs.append(obj)
    logs = []
    failed = False
    for s, p in procs:
        out, _ = p.communicate()
        logs.append(f"== {s}\n{out}")
        if p.returncode != 0:
            failed = True
    if failed or verbose:
        sys.stderr.write("\n".join(logs))
    if failed:
        raise RuntimeError("nvcc failed")
    tmp = LIB + ".tmp"
    cmd = [nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp, *objs,
           "-Xlinker", "--no-undefined", "-lrt", "-ldl", "-lpthread"]
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout)
        raise RuntimeError("link failed")
    os.replace(tmp, LIB)
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--verbose", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, verbose=a.verbose))


if __name__ == "__main__":
    main()
