"""Build libw4.so in-tree with nvcc for sm_103a (no cmake), and the binding's
extension module w4_host.so beside it.

The translation units compile in parallel; both land in
int4_weight_mixed_gb300/_build/.  libw4 knows nothing of torch or Python; the
extension module links against it and torch's libraries.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libw4.so")
HOST = os.path.join(BUILD, "w4_host.so")
HOST_STAMP = os.path.join(BUILD, "w4_host.for")  # the torch and Python it was built for
HOST_SOURCE = os.path.join(CSRC, "w4_host.cpp")
SOURCES = ["w4_api.cu", "w4_kernels.cu", "w4_tc.cu", "w4_tc2.cu", "w4_tc3.cu", "w4_dk.cu", "w4_noalloc.cu",
           "w4_ds.cu", "w4_quant.cu", "w4_gv.cu", "w4_norm.cu",
           "w4_tc_ep.cu", "w4_tc_ep2.cu", "w4_cache.cu", "w4_attn.cu", "w4_attn_dec.cu", "w4_attn_tc.cu"]
HEADERS = ["w4_internal.h", "w4_ptx.cuh", "w4_tc_kernel.cuh", "w4_epilogue.cuh", "w4_quant.cuh", "w4_cache.cuh", "w4_attn_plan.cuh", "w4_attn_math.cuh", os.path.join("..", "..", "include", "w4.h")]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build libw4")
    return cand


def _newest(paths) -> float:
    return max(os.path.getmtime(p) for p in paths)


def _host_key() -> str:
    """The extension module is compiled against torch's C++ classes: it is good
    for the torch and the Python it was built with alone."""
    import torch
    return f"torch {torch.__version__}, {sys.implementation.cache_tag}"


def host_lacks() -> str:
    """What keeps the built extension module from being loaded, or ""."""
    if not os.path.exists(HOST):
        return f"is not built (no {HOST})"
    try:
        with open(HOST_STAMP) as f:
            built = f.read()
    except OSError:
        built = "an unknown torch"
    return "" if built == _host_key() else f"was built for {built}, this is {_host_key()}"


def _torch_dir() -> str:
    import torch
    return os.path.dirname(torch.__file__)


def _host_compile(nvcc: str, obj: str) -> list:
    inc = os.path.join(_torch_dir(), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-Wall",
            "-I" + sysconfig.get_paths()["include"], "-isystem", inc,
            "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda,
            "-c", HOST_SOURCE, "-o", obj]


def _host_link(obj: str, out: str) -> list:
    lib = os.path.join(_torch_dir(), "lib")
    return [shutil.which("g++") or "g++", "-shared", "-o", out, obj, "-L" + BUILD, "-l:libw4.so",
            "-Wl,-rpath,$ORIGIN", "-L" + lib, "-Wl,-rpath," + lib, "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch", "-ltorch_python"]


def _run(jobs, verbose: bool) -> None:
    """Runs the compiler commands (name, command) side by side."""
    procs = []
    for src, cmd in jobs:
        if verbose:
            print(" ".join(cmd))
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    errors = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            errors.append(f"{src}:\n{out.decode(errors='replace')}")
    if errors:
        raise RuntimeError("libw4 build failed\n" + "\n".join(errors))


def build(force: bool = False, verbose: bool = False) -> str:
    headers = [os.path.join(CSRC, h) for h in HEADERS]
    sources = [os.path.join(CSRC, s) for s in SOURCES]
    fresh = lambda out, inputs: (not force and os.path.exists(out) and
                                 os.path.getmtime(out) >= _newest(inputs))
    lib = fresh(LIB, sources + headers)
    host = fresh(HOST, headers + [HOST_SOURCE]) and not host_lacks()
    if lib and host:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    objs = [os.path.join(BUILD, s.replace(".cu", ".o")) for s in SOURCES]
    host_obj = os.path.join(BUILD, "w4_host.o")
    jobs = []
    if not host:
        jobs.append(("w4_host.cpp", _host_compile(nvcc, host_obj)))
    if not lib:
        jobs += [(s, [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, s), "-o", o])
                 for s, o in zip(SOURCES, objs)]
    _run(jobs, verbose)
    if not lib:
        tmp = LIB + ".tmp.%d" % os.getpid()
        subprocess.check_call([nvcc, *ARCH, "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    if not host:
        if os.path.exists(HOST_STAMP):
            os.remove(HOST_STAMP)
        tmp = HOST + ".tmp.%d" % os.getpid()
        subprocess.check_call(_host_link(host_obj, tmp))
        os.replace(tmp, HOST)
        with open(HOST_STAMP, "w") as f:
            f.write(_host_key())
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
