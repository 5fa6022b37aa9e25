"""Build libbeam_moe.so in-tree with nvcc for sm_100a (cross-compiles without a GPU), and the native
side of training.py, _training.so, with g++ against the installed torch."""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import re
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libbeam_moe.so")
UNITS = [os.path.join(CSRC, f) for f in ("beam_moe.cu", "train_ops.cu")]
OBJ = os.path.join(HERE, "_build")
BINDING_SRC = os.path.join(CSRC, "binding.cpp")
BINDING = os.path.join(HERE, "_training.so")
BINDING_ABI = os.path.join(OBJ, "_training.abi")   # binding_abi() when BINDING was built
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

NVCC_FLAGS = [
    "-O3", "-std=c++17", "-lineinfo",
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-Xcompiler", "-fPIC",
    "-I", os.path.join(ROOT, "include"),
]


def sources():
    out = [os.path.join(ROOT, "include", "beam_moe.h")]
    for f in sorted(os.listdir(CSRC)):
        if f.endswith((".cu", ".cuh", ".h")):
            out.append(os.path.join(CSRC, f))
    return out


def _older(target: str, files) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in files)


def binding_abi() -> str:
    """What the native module is built against: the installed torch and this Python."""
    return f"torch {importlib.metadata.version('torch')} {sysconfig.get_config_var('EXT_SUFFIX')}"


def _binding_stale() -> bool:
    if _older(BINDING, _included(BINDING_SRC)) or not os.path.exists(BINDING_ABI):
        return True
    with open(BINDING_ABI) as f:
        return f.read() != binding_abi()


def stale() -> bool:
    return _older(LIB, sources()) or _binding_stale()


def binding_command(out: str) -> list:
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    cuda = os.path.dirname(os.path.dirname(NVCC))
    inc = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    libs = ("torch_python", "torch", "torch_cpu", "torch_cuda", "c10", "c10_cuda", "dl")
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            *[a for p in inc for a in ("-isystem", p)], "-o", out, BINDING_SRC,
            "-L", os.path.join(torch, "lib"), *["-l" + n for n in libs]]


def _included(unit: str):
    """The headers a unit includes, directly or through another header, and the unit itself."""
    todo, seen = [unit], set()
    while todo:
        f = todo.pop()
        if f in seen or not os.path.exists(f):
            continue
        seen.add(f)
        for name in re.findall(r'^#include "([^"]+)"', open(f).read(), re.M):
            todo.append(os.path.normpath(os.path.join(CSRC, name)))
    return sorted(seen)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the units whose sources changed (side by side), then link the library."""
    if not force and not stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    jobs, objs = [], []
    for unit in UNITS:
        obj = os.path.join(OBJ, os.path.basename(unit)[:-3] + ".o")
        objs.append(obj)
        if not force and not _older(obj, _included(unit)):
            continue
        tmp = obj + f".tmp{os.getpid()}"
        cmd = [NVCC, *NVCC_FLAGS, "-c", "-o", tmp, unit]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
            print(" ".join(cmd), flush=True)
        jobs.append((subprocess.Popen(cmd), cmd, tmp, obj))
    binding = force or _binding_stale()
    if binding:
        tmp = BINDING + f".tmp{os.getpid()}"
        cmd = binding_command(tmp)
        jobs.append((subprocess.Popen(cmd), cmd, tmp, BINDING))
    failed = [cmd for proc, cmd, _, _ in jobs if proc.wait() != 0]
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    for _, _, tmp, obj in jobs:
        os.replace(tmp, obj)
    if binding:
        tmp = BINDING_ABI + f".tmp{os.getpid()}"
        with open(tmp, "w") as f:
            f.write(binding_abi())
        os.replace(tmp, BINDING_ABI)
    if not force and not _older(LIB, objs):
        return LIB
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.check_call([NVCC, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp, *objs])
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
