"""Builds ``libgptq.so`` (the C-ABI CUDA library) in-tree with nvcc for sm_103a, and ``_marshal.so``
(the compiled part of the Python binding, against torch's headers).

Each ``csrc/*.cu`` translation unit is compiled in parallel into ``_build/``, then linked
into ``post_weight_quantization_03_gb300/libgptq.so``; ``csrc/marshal.cpp`` likewise.  Each is rebuilt
only when one of its sources or headers is newer, ``_marshal.so`` also for another torch or Python.
The library needs nvcc alone: without g++ or torch ``_marshal.so`` is left out, and the helpers that
need it say so.  Usage: ``python -m post_weight_quantization_03_gb300.build_lib``.
"""

from __future__ import annotations

import glob
import importlib.util
import os
import re
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
MARSHAL_TAG = os.path.join(BUILD, "marshal.tag")   # what _marshal.so was built against
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


def _newer(target, inputs) -> bool:
    """``target`` is there and newer than its inputs."""
    if not os.path.exists(target):
        return False
    t = os.path.getmtime(target)
    return all(os.path.getmtime(p) <= t for p in [*inputs, os.path.abspath(__file__)])


def _headers():
    return glob.glob(os.path.join(INCLUDE, "*.h"))


def library_up_to_date() -> bool:
    return _newer(LIB, _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + _headers())


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return list(spec.submodule_search_locations)[0] if spec is not None else None


def _cxx():
    return os.environ.get("CXX") or shutil.which("g++")


def marshal_tag():
    """The torch and the Python whose C++ classes and ABI ``_marshal.so`` has to be built against."""
    torch = _torch_dir()
    if torch is None:
        return None
    with open(os.path.join(torch, "version.py")) as f:
        version = re.search(r"^__version__ = ['\"](.*)['\"]", f.read(), re.MULTILINE)
    return f"torch {version.group(1) if version else '?'}, {sysconfig.get_config_var('SOABI')}"


def marshal_built_against():
    """What ``_marshal.so`` was built against, as ``marshal_tag`` has it; None where that is not known."""
    if not os.path.exists(MARSHAL) or not os.path.exists(MARSHAL_TAG):
        return None
    with open(MARSHAL_TAG) as f:
        return f.read()


def marshal_up_to_date() -> bool:
    return _newer(MARSHAL, [os.path.join(CSRC, "marshal.cpp"), *_headers()]) and marshal_built_against() == marshal_tag()


def up_to_date() -> bool:
    """Nothing of what can be built here is left to build."""
    return library_up_to_date() and (marshal_up_to_date() or _torch_dir() is None or not _cxx())


def _marshal_commands(nvcc, obj, out):
    """Compiler and linker calls of ``_marshal.so``."""
    cxx, torch = _cxx(), _torch_dir()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))
    include = [os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(torch, "lib")
    return ([cxx, "-O2", "-std=c++17", "-fPIC", *(f"-I{p}" for p in include), "-c", os.path.join(CSRC, "marshal.cpp"),
             "-o", obj],
            [cxx, "-shared", "-o", out, obj, f"-L{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10",
             f"-Wl,-rpath,{lib}"])


def _start(cmd, verbose=False):
    if verbose:
        print(" ".join(cmd), flush=True)
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)


def _finish(procs, verbose=False):
    """Waits for compilers and linkers (name, process); raises with the output of those that failed."""
    failed = []
    for name, p in procs:
        out, _ = p.communicate()
        if verbose and out:
            print(out.decode(errors="replace"), flush=True)
        if p.returncode != 0:
            failed.append(f"--- {name}\n{out.decode(errors='replace')}")
    if failed:
        raise RuntimeError("build failed:\n" + "\n".join(failed))


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile and link what is not up to date; returns the library's path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    marshal = []
    if (force or not marshal_up_to_date()) and _torch_dir() is not None and _cxx():
        compile_marshal, link_marshal = _marshal_commands(nvcc, os.path.join(BUILD, "marshal.o"), MARSHAL + ".tmp")
        marshal.append(("marshal.cpp", _start(compile_marshal, verbose)))
    try:
        if force or not library_up_to_date():
            procs, objs = [], []
            for src in _sources():
                obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
                objs.append(obj)
                procs.append((src, _start([nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", src, "-o", obj], verbose)))
            _finish(procs, verbose)
            tmp = LIB + ".tmp"
            _finish([(LIB, _start([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "shared",
                                   "-Xlinker", "-rpath,/usr/local/cuda/lib64"], verbose))], verbose)
            os.replace(tmp, LIB)
    finally:
        # (the library is in place before anything of the marshalling can fail)
        _finish(marshal, verbose)
    if marshal:
        _finish([(MARSHAL, _start(link_marshal, verbose))], verbose)
        if os.path.exists(MARSHAL_TAG):
            os.remove(MARSHAL_TAG)   # (never one of another build)
        os.replace(MARSHAL + ".tmp", MARSHAL)
        with open(MARSHAL_TAG, "w") as f:
            f.write(marshal_tag())
    return LIB


if __name__ == "__main__":
    force = "--force" in sys.argv
    extra = ["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else []
    print(build(force=force, verbose=True, extra_flags=extra))
