"""Builds libmoe.so in-tree with nvcc for sm_103a (no cmake, no torch
extension machinery): one nvcc per translation unit, run in parallel, then a
shared-library link against the shared CUDA runtime."""
from __future__ import annotations

import os
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor
from typing import List, Optional

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe.so")
# Checked build: every row index read from a routing table is verified against
# its buffer before use (MOE_ECORRUPT); a separate library and object folder.
BUILD_CHECKED = os.path.join(PKG, "_build_checked")
LIB_CHECKED = os.path.join(PKG, "libmoe_checked.so")
# The CPython modules of ffn.py and train.py: argument checks on torch tensors, calls into
# libmoe.so next to them.  Built against the installed torch, with the host compiler.
LIB_FFN = os.path.join(PKG, "_ffn.so")
STAMP_FFN = os.path.join(BUILD, "ffn.stamp")
LIB_TRAIN = os.path.join(PKG, "_train.so")
STAMP_TRAIN = os.path.join(BUILD, "train.stamp")
SOURCES = ["route_count.cu", "route_split.cu", "route_cluster.cu", "route_pack.cu", "route_pack_fp8.cu", "dispatch_pack.cu", "dispatch_fp8.cu", "dispatch_staged.cu", "dense_a2a.cu", "combine.cu", "combine_two_level.cu", "moe_abi.cu", "moe_noalloc.cu",
           "add_norm_fp8.cu", "expert_gemm.cu", "decode_layer.cu", "ffn_abi.cu",
           "router.cu", "route_grad.cu", "expert_linear.cu", "expert_linear_few.cu", "train_abi.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe.so")


def _cuda_lib_dir(nv: str) -> str:
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nv))), "lib64")


def _newest_input() -> float:
    paths = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE)]
    return max(os.path.getmtime(p) for p in paths)


def _read(path: str) -> Optional[str]:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return None


def build(force: bool = False, verbose: bool = False, extra_flags: Optional[List[str]] = None,
          checked: bool = False) -> str:
    """Compile csrc/*.cu into libmoe.so next to this file (libmoe_checked.so
    with checked=True); returns its path."""
    lib = LIB_CHECKED if checked else LIB
    build_dir = BUILD_CHECKED if checked else BUILD
    if not force and os.path.exists(lib) and os.path.getmtime(lib) >= _newest_input() and not extra_flags:
        return lib
    nv = nvcc()
    os.makedirs(build_dir, exist_ok=True)
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler",
                    "-fvisibility=hidden", "-I", INCLUDE, "-I", CSRC] + list(extra_flags or [])
    if checked:
        flags.append("-DMOE_CHECKED")

    def compile_one(src: str) -> str:
        obj = os.path.join(build_dir, src.replace(".cu", ".o"))
        cmd = [nv] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = lib + f".tmp{os.getpid()}"
    libdir = _cuda_lib_dir(nv)
    cmd = [nv] + ARCH + ["-shared", "-cudart", "shared", "-Xlinker", f"-soname={os.path.basename(lib)}", "-o", tmp] + objs + [
        "-Xlinker", f"-rpath,{libdir}", "-L", libdir]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of {os.path.basename(lib)} failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    return lib


def _build_module(source: str, lib: str, stamp: str, force: bool) -> str:
    import sysconfig

    import torch
    src = os.path.join(CSRC, source)
    troot = os.path.dirname(torch.__file__)
    # What the module was compiled against: another torch or Python needs another module.
    against = f"torch {torch.__version__} in {troot}, {sysconfig.get_config_var('SOABI')}\n"
    if not force and os.path.exists(lib) and os.path.getmtime(lib) >= _newest_input() and _read(stamp) == against:
        return lib
    build()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-shared", "-fvisibility=hidden", src, "-o", tmp]
    for inc in (INCLUDE, os.path.join(troot, "include"), os.path.join(troot, "include", "torch", "csrc", "api", "include"),
                sysconfig.get_paths()["include"], os.path.join(cuda, "include")):
        cmd += ["-I", inc]
    tlib = os.path.join(troot, "lib")
    cmd += [LIB, "-L", tlib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-L", os.path.join(cuda, "lib64"), "-lcudart",
            "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{tlib}", f"-Wl,-rpath,{os.path.join(cuda, 'lib64')}"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {source}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, lib)
    os.makedirs(BUILD, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(against)
    return lib


def build_ffn(force: bool = False) -> str:
    """Compile csrc/ffn_py.cc into _ffn.so next to libmoe.so; returns its path."""
    return _build_module("ffn_py.cc", LIB_FFN, STAMP_FFN, force)


def build_train(force: bool = False) -> str:
    """Compile csrc/train_py.cc into _train.so next to libmoe.so; returns its path."""
    return _build_module("train_py.cc", LIB_TRAIN, STAMP_TRAIN, force)


if __name__ == "__main__":
    print(build(force=True, verbose=True))
    print(build_ffn(force=True))
    print(build_train(force=True))
