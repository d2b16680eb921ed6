"""Builds libvdtq.so in-tree with hipcc for gfx950.

    python -m video_diffusion_transformer_block_amd.build

Floating-point flags are part of the contract: no contraction (the
Hadamard butterflies and the quantization steps are bit-exact fp32 sequences),
correctly rounded fp32 division, fp32 denormals kept (the HIP default), and
no compiler-formed packed-fp32 instructions.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(HERE, "libvdtq.so")
# plain streaming passes the benchmark times as ceilings (not the library's ABI)
BENCH_LIB = os.path.join(HERE, "libvdtq_bench.so")
BENCH_SOURCES = ["bench_stream.hip"]
SOURCES = ["hadamard_quantize.hip", "qgemm.hip", "qgemm_mx.hip", "qgemm_w4a16.hip", "block_stats.hip",
           "rmsnorm_quantize.hip", "qgemv.hip", "qgemm_mx_grouped.hip", "api.cpp", "dmpq.cpp"]

# the Python entry of the short calls (torch's C++ interface; links LIB)
FAST = os.path.join(HERE, "_fastcalls.so")
FAST_SOURCE = "fast_calls.cpp"

HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
ROCM = os.environ.get("ROCM_PATH", "/opt/rocm")
CXX = os.environ.get("CXX", shutil.which("g++") or "c++")
ARCH = "gfx950"
FLAGS = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
         "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
         "-fno-gpu-flush-denormals-to-zero",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-function", "-I", os.path.join(ROOT, "include")]


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
    lang = ["-x", "hip"] if src.endswith(".cpp") else []
    cmd = [HIPCC, *FLAGS, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link(objs, out: str) -> None:
    tmp = out + ".tmp"
    cmd = [HIPCC, "-shared", f"--offload-arch={ARCH}", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _compile_fast() -> str:
    """The host-only module: compiled as plain C++ against torch's headers."""
    import sysconfig
    import torch
    from torch.utils.cpp_extension import include_paths
    obj = os.path.join(BUILD, "fast_calls.o")
    inc = [a for p in (*include_paths(), sysconfig.get_paths()["include"], os.path.join(ROCM, "include"))
           for a in ("-isystem", p)]
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function", "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc, "-c",
           os.path.join(CSRC, FAST_SOURCE), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{CXX} failed for {FAST_SOURCE}:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_fast(obj: str) -> None:
    from torch.utils.cpp_extension import library_paths
    tmp = FAST + ".tmp"
    libs = [a for p in library_paths() for a in (f"-L{p}", f"-Wl,-rpath,{p}")]
    cmd = [CXX, "-shared", "-o", tmp, obj, f"-L{HERE}", "-l:libvdtq.so", "-Wl,-rpath,$ORIGIN", *libs, "-lc10", "-lc10_hip",
           "-ltorch_cpu", "-ltorch_hip", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, FAST)


def build(verbose: bool = False) -> str:
    os.makedirs(BUILD, exist_ok=True)
    srcs = SOURCES + BENCH_SOURCES
    with ThreadPoolExecutor(max_workers=min(len(srcs), 8)) as ex:
        fast = ex.submit(_compile_fast)
        objs = list(ex.map(_compile, srcs))
        fast_obj = fast.result()
    _link(objs[:len(SOURCES)], LIB)
    _link(objs[len(SOURCES):], BENCH_LIB)
    _link_fast(fast_obj)
    if verbose:
        print("built", LIB, "and", BENCH_LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
