"""Builds the CUDA library libabg.so in-tree with nvcc for sm_103a, and the
CPython module _marshal.so (the draft calls' arguments from torch tensors).

Each source under csrc/ is compiled to an object in parallel, then the objects
are linked into shared libraries next to this file.  Rebuilds only when a
source or header is newer than the libraries.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libabg.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I" + os.path.join(ROOT, "include")]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + [os.path.join(CSRC, "marshal.cpp")] + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(ROOT, "include", "*.h"))


def stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MARSHAL):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    return any(os.path.getmtime(p) > t for p in _deps() + [os.path.abspath(__file__)])


def _torch_dirs():
    import importlib.util
    root = os.path.dirname(importlib.util.find_spec("torch").origin)  # without importing it
    inc = os.path.join(root, "include")
    return [inc, os.path.join(inc, "torch", "csrc", "api", "include")], os.path.join(root, "lib")


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    procs = []
    objs = []
    for src in _sources():
        obj = os.path.join(OBJ, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [NVCC, *FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    marshal = os.path.join(CSRC, "marshal.cpp")
    marshal_obj = os.path.join(OBJ, "marshal.o")
    torch_inc, torch_lib = _torch_dirs()
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", marshal, "-o", marshal_obj, "-I" + sysconfig.get_paths()["include"],
           "-I" + cuda_inc] + ["-isystem" + d for d in torch_inc]
    if verbose:
        print(" ".join(cmd))
    procs.append((marshal, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
        elif verbose and out:
            print(out.decode(errors="replace"))
    if failed:
        raise RuntimeError("compilation failed:\n" + "\n".join(f"{s}:\n{o}" for s, o in failed))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([NVCC, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs], check=True)
    os.replace(tmp, LIB)
    # torch's own libraries are loaded by then (by name); libabg.so lies beside
    tmp = MARSHAL + f".tmp{os.getpid()}"
    subprocess.run(["g++", "-shared", "-o", tmp, marshal_obj, "-L" + HERE, "-l:libabg.so", "-Wl,-rpath,$ORIGIN",
                    "-L" + torch_lib, "-ltorch_python", "-lc10_cuda", "-lc10", "-ltorch_cpu"], check=True)
    os.replace(tmp, MARSHAL)
    return LIB


if __name__ == "__main__":
    build(force=True, verbose=True)
