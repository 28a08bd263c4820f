"""Builds ``libgptq.so`` (the C-ABI CUDA library) in-tree with nvcc for sm_103a, and ``_marshal.so``
(the compiled part of the Python binding, against torch's headers).

Each ``csrc/*.cu`` translation unit is compiled in parallel into ``_build/``, then linked
into ``post_weight_quantization_03_gb300/libgptq.so``; ``csrc/marshal.cpp`` likewise.  Rebuilds only
when a source or header is newer than both.  Usage: ``python -m
post_weight_quantization_03_gb300.build_lib``.
"""

from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgptq.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-I", INCLUDE]


def _nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libgptq.so")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _inputs():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(CSRC, "marshal.cpp")] + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + [os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(MARSHAL):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(MARSHAL))
    return all(os.path.getmtime(p) <= t for p in _inputs())


def _marshal_commands(nvcc, obj, out):
    """Compiler and linker calls of ``_marshal.so``."""
    cxx = os.environ.get("CXX") or shutil.which("g++")
    spec = importlib.util.find_spec("torch")
    if not cxx or spec is None:
        raise RuntimeError("g++ and torch are required to build _marshal.so")
    torch = list(spec.submodule_search_locations)[0]
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(torch, "lib")
    return ([cxx, "-O2", "-std=c++17", "-fPIC", *(f"-I{p}" for p in include), "-c", os.path.join(CSRC, "marshal.cpp"),
             "-o", obj],
            [cxx, "-shared", "-o", out, obj, f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
             f"-Wl,-rpath,{lib}"])


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link the library; returns its path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    marshal_obj = os.path.join(BUILD, "marshal.o")
    compile_marshal, link_marshal = _marshal_commands(nvcc, marshal_obj, MARSHAL + ".tmp")
    procs = [(compile_marshal[-3], subprocess.Popen(compile_marshal, stdout=subprocess.PIPE,
                                                    stderr=subprocess.STDOUT))]
    objs = []
    for src in _sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                            stderr=subprocess.STDOUT)))
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        if verbose and out:
            print(out.decode(errors="replace"), flush=True)
        if p.returncode != 0:
            failed.append((src, out.decode(errors="replace")))
    if failed:
        msg = "\n".join(f"--- {s}\n{o}" for s, o in failed)
        raise RuntimeError(f"nvcc failed:\n{msg}")
    tmp = LIB + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "shared",
           "-Xlinker", "-rpath,/usr/local/cuda/lib64"]
    if verbose:
        print(" ".join(cmd), flush=True)
    for link in (cmd, link_marshal):
        r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(MARSHAL + ".tmp", MARSHAL)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force=force, verbose=True, extra_flags=extra))
