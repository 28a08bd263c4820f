"""The build's two parts: the C library needs nvcc alone, the binding's compiled part also g++ and torch, and is
built again for another torch.  (Compilers are stand-ins that write their output's name into it.)"""

import os

import pytest

from post_weight_quantization_03_gb300 import build_lib, gptq

COMPILER = """#!/bin/sh
echo "$@" >> "{log}"
[ -e "{log}.fails" ] && exit 1
while [ $# -gt 0 ]; do [ "$1" = -o ] && echo "$2" > "$2"; shift; done
exit 0
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """build_lib on a tree of its own, with stand-ins for nvcc, g++ and torch."""
    for sub in ("csrc", "include", "_build", "torch"):
        (tmp_path / sub).mkdir()
    for name in ("csrc/a.cu", "csrc/b.cu", "csrc/common.cuh", "csrc/marshal.cpp", "include/gptq.h"):
        (tmp_path / name).write_text("")
    (tmp_path / "torch" / "version.py").write_text("__version__ = '1.0'\n")
    for name in ("nvcc", "g++"):
        (tmp_path / name).write_text(COMPILER.format(log=tmp_path / f"{name}.log"))
        (tmp_path / name).chmod(0o755)
    for name, at in (("CSRC", "csrc"), ("BUILD", "_build"), ("INCLUDE", "include"), ("LIB", "libgptq.so"), ("MARSHAL", "_marshal.so"),
                     ("MARSHAL_TAG", "_build/marshal.tag")):
        monkeypatch.setattr(build_lib, name, str(tmp_path / at))
    monkeypatch.setenv("NVCC", str(tmp_path / "nvcc"))
    monkeypatch.setenv("CXX", str(tmp_path / "g++"))

    class Spec:
        submodule_search_locations = [str(tmp_path / "torch")]

    monkeypatch.setattr(build_lib.importlib.util, "find_spec", lambda name: Spec() if name == "torch" else None)
    monkeypatch.setattr(build_lib, "__file__", str(tmp_path / "csrc" / "a.cu"))
    return tmp_path


def _calls(tree, name):
    log = tree / f"{name}.log"
    lines = log.read_text().splitlines() if log.exists() else []
    if log.exists():
        log.unlink()
    return len(lines)


def test_builds_both_and_only_what_is_older(tree):
    assert build_lib.build() == str(tree / "libgptq.so")
    assert (tree / "_marshal.so").exists() and _calls(tree, "nvcc") == 3 and _calls(tree, "g++") == 2
    build_lib.build()
    assert _calls(tree, "nvcc") == 0 and _calls(tree, "g++") == 0
    later = os.path.getmtime(tree / "_marshal.so") + 10
    os.utime(tree / "csrc" / "marshal.cpp", (later, later))
    assert not build_lib.up_to_date()
    build_lib.build()
    assert _calls(tree, "nvcc") == 0 and _calls(tree, "g++") == 2
    os.utime(tree / "csrc" / "marshal.cpp", (0, 0))
    os.utime(tree / "csrc" / "common.cuh", (later, later))
    build_lib.build()
    assert _calls(tree, "nvcc") == 3 and _calls(tree, "g++") == 0


@pytest.mark.parametrize("lacks", ["torch", "g++"])
def test_the_library_needs_nvcc_alone(tree, monkeypatch, lacks):
    if lacks == "torch":
        monkeypatch.setattr(build_lib.importlib.util, "find_spec", lambda name: None)
    else:
        monkeypatch.delenv("CXX")
        monkeypatch.setattr(build_lib.shutil, "which", lambda name: None)
    build_lib.build()
    assert (tree / "libgptq.so").exists() and not (tree / "_marshal.so").exists() and build_lib.up_to_date()
    assert _calls(tree, "nvcc") == 3


def test_a_marshalling_that_does_not_compile_leaves_the_library(tree):
    (tree / "g++.log.fails").write_text("")
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        build_lib.build()
    assert (tree / "libgptq.so").exists() and not (tree / "_marshal.so").exists() and not build_lib.up_to_date()
    (tree / "g++.log.fails").unlink()
    _calls(tree, "nvcc")
    build_lib.build()
    assert _calls(tree, "nvcc") == 0 and build_lib.up_to_date()


def test_a_library_that_does_not_compile(tree):
    (tree / "nvcc.log.fails").write_text("")
    with pytest.raises(RuntimeError, match="a.cu"):
        build_lib.build()
    assert not (tree / "libgptq.so").exists()


def test_another_torch(tree, monkeypatch):
    build_lib.build()
    _calls(tree, "nvcc"), _calls(tree, "g++")
    (tree / "torch" / "version.py").write_text("__version__ = '1.1'\n")
    assert build_lib.library_up_to_date() and not build_lib.up_to_date()
    # one of another torch is not loaded
    monkeypatch.setattr(gptq, "_MARSHAL", None)
    monkeypatch.setattr(gptq, "load", lambda: None)
    with pytest.raises(RuntimeError, match="built against torch 1.0"):
        gptq._marshal()
    build_lib.build()
    assert _calls(tree, "nvcc") == 0 and _calls(tree, "g++") == 2 and build_lib.up_to_date()
    (tree / "_marshal.so").unlink()
    with pytest.raises(RuntimeError, match="missing"):
        gptq._marshal()
