"""Build libstrata_moe.so (HIP, gfx950) in-tree with hipcc."""
from __future__ import annotations

import concurrent.futures as cf
import os
import subprocess
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libstrata_moe.so")
SOURCES = ["api.hip", "popularity.hip", "route.hip", "gemv.hip", "gemv_gu3.hip", "gemv_gu2.hip", "gemv_dn3.hip", "gemv_dn2.hip",
           "gemm.hip", "gemm_gu3.hip", "gemm_gu2.hip", "gemm_dn3.hip", "gemm_dn2.hip", "combine.hip",
           "probe.hip", "sort.hip", "rows.hip", "block_norm.hip", "block_norm_any.hip",
           *(f"block_norm_{x}{y}{u}.hip" for x in "fh" for y in "fh" for u in "fh"), "grouped.hip",
           "balance.hip", "embed.hip", "vocab.hip", "orth.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
# Packed fp32 VALU forms are disabled for every kernel in this library.
FLAGS = ["-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC", "-Wall", "-Wno-unused-function",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", os.path.join(HERE, "..", "include")]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


# The host consumer of the miss list: one object per instruction set (the
# library picks one at run time), built by the host compiler.
HOST_SOURCE = "host_experts.cpp"
HOST_ISAS = {"hx512": ["-mavx512f", "-mavx512bw", "-mavx512dq", "-mavx512vl", "-mfma"],
             "hx256": ["-mavx2", "-mfma"]}
CXX = os.environ.get("CXX_HOST", "g++")


def _compile_host(ns: str) -> str:
    obj = os.path.join(BUILD, f"host_experts_{ns}.o")
    cmd = [CXX, "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-psabi", *HOST_ISAS[ns], f"-DHX_NS={ns}",
           "-I", os.path.join(HERE, "..", "include"),
           "-c", os.path.join(CSRC, HOST_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"host compile failed for {ns}:\n{r.stdout}\n{r.stderr}")
    return obj


def _compile_host_common() -> str:
    obj = os.path.join(BUILD, "host.o")
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-Wall", "-pthread", "-I", os.path.join(HERE, "..", "include"),
           "-c", os.path.join(CSRC, "host.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"host compile failed for host.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


# The operators' tensor checks: a CPython module against torch's headers.
BINDING = os.path.join(HERE, "_binding.so")


def _compile_binding() -> str:
    import sysconfig
    try:
        import torch
    except (ImportError, OSError):   # the operators' binding is for torch's tensors
        return ""
    base = os.path.dirname(torch.__file__)
    tmp = BINDING + ".tmp"
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", os.path.join(HERE, "..", "include"), "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"], os.path.join(CSRC, "binding.cpp"), "-o", tmp,
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"host compile failed for binding.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, BINDING)
    return BINDING


def build(verbose: bool = False) -> str:
    """Compile every source (always), link the shared library and the binding's module.

    The library needs neither Python's headers nor torch's: where the module
    does not compile against them the library is built all the same, with a
    warning, and the operators say so when they are called from Python.
    """
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=8) as ex:
        futs = [ex.submit(_compile, src) for src in SOURCES]
        futs += [ex.submit(_compile_host, ns) for ns in HOST_ISAS]
        futs.append(ex.submit(_compile_host_common))
        binding = ex.submit(_compile_binding)
        objs = [f.result() for f in futs]
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs, "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    if binding.exception() is not None:
        if os.path.exists(BINDING):   # of an earlier build: its calls need not fit this library
            os.remove(BINDING)
        warnings.warn(f"the operators cannot be called from Python: {binding.exception()}", RuntimeWarning)
    if verbose:
        print("built", LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
