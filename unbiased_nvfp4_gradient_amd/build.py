"""Build libnvfp4.so (gfx950) in-tree with hipcc, and _tensors.so, the reader of tensor lists, with
the host compiler.

Every HIP source is compiled with -ffp-contract=off (the quantizer's arithmetic is fixed in
binary32 with one rounding per operation) and without packed-FP32 instructions.
"""
from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libnvfp4.so")
BUILD_DIR = os.path.join(PKG, "_build")

SOURCES = ["nvfp4_kernels.hip", "nvfp4_gemm.hip", "nvfp4_api.cpp", "train_norm.hip",
           "train_ce.hip", "train_ce_few.hip", "train_clip.hip", "train_api.cpp"]

TENSORS_SOURCE = "train_tensors.cpp"
TENSORS = os.path.join(PKG, "_tensors.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
COMMON = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-ffp-contract=off",
    "-fno-fast-math", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-I", INCLUDE,
]


def _tensors_command(out: str):
    """Host compiler command of the tensor list reader: a Python module against torch's headers."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    includes = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *(f"-isystem{i}" for i in includes), os.path.join(CSRC, TENSORS_SOURCE), "-o", out,
            f"-L{libs}", "-ltorch_python", "-ltorch_cpu", "-lc10", f"-Wl,-rpath,{libs}"]


def build(verbose: bool = False) -> str:
    """Compile every source to an object in parallel, then link the shared library."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = []
    objs = []
    cmds = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, os.path.splitext(src)[0] + ".o")
        objs.append(obj)
        cmds.append((src, [HIPCC, *COMMON, "-c", os.path.join(CSRC, src), "-o", obj]))
    cmds.append((TENSORS_SOURCE, _tensors_command(TENSORS + ".tmp")))
    for src, cmd in cmds:
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, cwd=BUILD_DIR, stdout=subprocess.PIPE,
                                            stderr=subprocess.STDOUT, text=True)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out))
        elif verbose and out.strip():
            print(out, flush=True)
    if failed:
        for src, out in failed:
            sys.stderr.write(f"--- the compiler failed on {src}\n{out}\n")
        raise RuntimeError("libnvfp4 build failed: " + ", ".join(s for s, _ in failed))
    tmp = LIB + ".tmp"
    subprocess.check_call([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs],
                          cwd=BUILD_DIR)
    os.replace(tmp, LIB)
    os.replace(TENSORS + ".tmp", TENSORS)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
