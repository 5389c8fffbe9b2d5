"""Builds the CUDA library libabg.so in-tree with nvcc for sm_103a, and the
CPython module _marshal.so (the draft calls' arguments from torch tensors).

Each source under csrc/ is compiled to an object in parallel, then the objects
are linked into shared libraries next to this file.  Each is rebuilt only when a
source or header of its own is newer than it.  The library needs neither torch
nor the module: without torch only the library is built, and an error in the
module's build comes after the library is in place.
"""
from __future__ import annotations

import glob
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libabg.so")
MARSHAL = os.path.join(HERE, "_marshal.so")
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "-I" + os.path.join(ROOT, "include")]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _headers():
    return glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _headers()


def _older(path, deps) -> bool:
    """Whether path is missing or older than one of deps."""
    if not os.path.exists(path):
        return True
    t = os.path.getmtime(path)
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def stale() -> bool:
    """Whether libabg.so has to be built."""
    return _older(LIB, _deps())


def marshal_stale() -> bool:
    """Whether _marshal.so has to be built (never without torch): also where it was
    built for another torch or Python."""
    return _torch_root() is not None and (_older(MARSHAL, [os.path.join(CSRC, "marshal.cpp")] + _headers()) or
                                          _built_for() not in (None, _host()))


def _host() -> str:
    """The Python and the torch that the module is compiled against."""
    version = os.path.join(_torch_root(), "version.py")
    text = ""
    if os.path.exists(version):
        with open(version) as f:
            text = f.read()
    return f"{sys.implementation.cache_tag} {_torch_root()}\n{text}"


def _built_for():
    """What _host() was when the module was linked (None: not known)."""
    note = os.path.join(OBJ, "marshal.host")
    if not os.path.exists(note):
        return None
    with open(note) as f:
        return f.read()


def _torch_root():
    """torch's folder, without importing it; None where there is no torch."""
    import importlib.util
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _start(cmd, verbose):
    if verbose:
        print(" ".join(cmd))
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish(procs, verbose):
    """Waits for compilers; raises what the ones that failed say."""
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if p.returncode != 0:
            failed.append(f"{src}:\n{out.decode(errors='replace')}")
        elif verbose and out:
            print(out.decode(errors="replace"))
    if failed:
        raise RuntimeError("compilation failed:\n" + "\n".join(failed))


def _start_marshal(verbose):
    root = _torch_root()
    src, obj = os.path.join(CSRC, "marshal.cpp"), os.path.join(OBJ, "marshal.o")
    inc = os.path.join(root, "include")
    cuda_inc = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    cmd = [CXX, "-O2", "-std=c++17", "-fPIC", "-c", src, "-o", obj, "-I" + sysconfig.get_paths()["include"],
           "-I" + cuda_inc, "-isystem" + inc, "-isystem" + os.path.join(inc, "torch", "csrc", "api", "include")]
    return [(src, _start(cmd, verbose))]


def _link_marshal():
    # torch's own libraries are loaded by then (by name); libabg.so lies beside
    tmp = MARSHAL + f".tmp{os.getpid()}"
    subprocess.run([CXX, "-shared", "-o", tmp, os.path.join(OBJ, "marshal.o"), "-L" + os.path.dirname(LIB), "-l:libabg.so",
                    "-Wl,-rpath,$ORIGIN", "-L" + os.path.join(_torch_root(), "lib"), "-ltorch_python", "-lc10_cuda",
                    "-lc10", "-ltorch_cpu"], check=True)
    os.replace(tmp, MARSHAL)
    with open(os.path.join(OBJ, "marshal.host"), "w") as f:
        f.write(_host())


def build(force: bool = False, verbose: bool = False, marshal: bool = True) -> str:
    """Builds what is stale (or, with force, all): the library, and with `marshal`
    the module too where there is torch."""
    lib = force or stale()
    marshal = marshal and (marshal_stale() or (force and _torch_root() is not None))
    if not lib and not marshal:
        return LIB
    os.makedirs(OBJ, exist_ok=True)
    procs, objs = [], []
    for src in _sources() if lib else ():
        objs.append(os.path.join(OBJ, os.path.basename(src)[:-3] + ".o"))
        procs.append((src, _start([NVCC, *FLAGS, "-c", src, "-o", objs[-1]], verbose)))
    beside = _start_marshal(verbose) if marshal else []
    try:
        _finish(procs, verbose)
        if lib:
            tmp = LIB + f".tmp{os.getpid()}"
            subprocess.run([NVCC, *ARCH, "-shared", "-cudart", "shared", "-o", tmp, *objs], check=True)
            os.replace(tmp, LIB)
    finally:
        if marshal:
            _finish(beside, verbose)
    if marshal:
        _link_marshal()
    return LIB


if __name__ == "__main__":
    build(force=True, verbose=True)
