"""Build libk3moe.so in-tree: every CUDA source compiled for sm_103a with nvcc; and
the binding's C++ part, _k3torch.so (csrc/torch_fast.cpp), against the installed torch.

Usage: ``python -m mxfp4_expert_ffn_router_gb300.build [--force]``.  Sources are
compiled in parallel into ``_build/`` and linked next to this file."""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
OUT = os.path.join(HERE, "libk3moe.so")
FAST = os.path.join(HERE, "_k3torch.so")
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["k3moe.cu", "route.cu", "bucket.cu", "ffn_gemv.cu", "ffn_gemm.cu", "combine.cu",
           "quant.cu", "k3moe_noalloc.cu", "router.cu", "expert_cache.cu", "rmsnorm.cu", "kv_cache.cu",
           "attn_decode.cu"]
NVCC = os.environ.get("NVCC", "nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                "-I", INCLUDE]


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files += [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    files.append(os.path.abspath(__file__))
    return files


def _fast_command(out: str) -> list:
    import sysconfig
    import torch
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I", inc, "-I", sysconfig.get_paths()["include"],
            "-I", cuda, os.path.join(CSRC, "torch_fast.cpp"), "-o", out, "-L", lib, "-ltorch_python", "-ltorch_cpu",
            "-lc10", "-lc10_cuda"]


def up_to_date() -> bool:
    if not os.path.exists(OUT) or not os.path.exists(FAST):
        return False
    t = min(os.path.getmtime(OUT), os.path.getmtime(FAST))
    return all(os.path.getmtime(f) <= t for f in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return OUT
    os.makedirs(BUILD_DIR, exist_ok=True)

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [NVCC] + FLAGS + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose:
            sys.stderr.write(r.stderr)
        return obj

    def compile_fast():
        tmp = FAST + f".tmp{os.getpid()}"
        r = subprocess.run(_fast_command(tmp), capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"g++ failed for torch_fast.cpp:\n{r.stdout}\n{r.stderr}")
        return tmp

    with ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 1)) as ex:
        fast = ex.submit(compile_fast)
        objs = list(ex.map(compile_one, SOURCES))
    tmp = OUT + f".tmp{os.getpid()}"
    r = subprocess.run([NVCC] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static"],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OUT)
    os.replace(fast.result(), FAST)
    return OUT


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(OUT)
