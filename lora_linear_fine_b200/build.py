"""Build the in-tree C-ABI library ``liblora_linear.so`` for sm_100a with nvcc,
and, with the host compiler, the torch functions' short way into it
(``_lora_torch``).

    python -m lora_linear_fine_b200.build            # build if sources changed
    python -m lora_linear_fine_b200.build --force    # always rebuild
    python -m lora_linear_fine_b200.build --ptxas-v  # also print register/smem usage
"""
from __future__ import annotations

import argparse
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "liblora_linear.so")
TORCH_SRC = os.path.join(CSRC, "lora_torch.cpp")
TORCH_MOD = os.path.join(PKG, "_lora_torch.so")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(INCLUDE, "*.h")))


def up_to_date() -> bool:
    if not os.path.exists(LIB):
        return False
    t = os.path.getmtime(LIB)
    return all(os.path.getmtime(s) <= t for s in sources())


def build(force: bool = False, ptxas_verbose: bool = False, quiet: bool = False) -> str:
    build_lib(force, ptxas_verbose, quiet)
    build_torch(force, quiet)
    return LIB


def build_lib(force: bool = False, ptxas_verbose: bool = False, quiet: bool = False) -> str:
    if not force and up_to_date():
        return LIB
    tmp = LIB + ".tmp"
    cmd = [nvcc(), *ARCH, "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
           "-Xcompiler", "-fPIC,-O2", "-shared", "-I", INCLUDE, "-I", CSRC,
           os.path.join(CSRC, "lora_linear.cu"), "-o", tmp]
    if ptxas_verbose:
        cmd.insert(1, "-Xptxas=-v")
    if not quiet:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, LIB)
    return LIB


def build_torch(force: bool = False, quiet: bool = False) -> str:
    """The torch module: bound to this interpreter's torch, linked with the library beside it."""
    newest = max(os.path.getmtime(p) for p in (TORCH_SRC, os.path.join(INCLUDE, "lora_linear.h"), __file__))
    if not force and os.path.exists(TORCH_MOD) and os.path.getmtime(TORCH_MOD) >= newest:
        return TORCH_MOD
    import torch
    from torch.utils import cpp_extension
    tmp = TORCH_MOD + ".tmp"
    paths = cpp_extension.include_paths("cuda") + [sysconfig.get_paths()["include"], INCLUDE]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-w",
           "-DTORCH_EXTENSION_NAME=_lora_torch", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           *(x for p in paths for x in ("-isystem", p)), TORCH_SRC, "-o", tmp,
           *(x for p in cpp_extension.library_paths("cuda") for x in ("-L", p)),
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", "-L", PKG, "-l:" + os.path.basename(LIB),
           "-Wl,-rpath,$ORIGIN"]
    if not quiet:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)
    os.replace(tmp, TORCH_MOD)
    return TORCH_MOD


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("--ptxas-v", action="store_true")
    a = ap.parse_args()
    print(build(force=a.force, ptxas_verbose=a.ptxas_v))


if __name__ == "__main__":
    main()
