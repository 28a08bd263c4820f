"""The library's per-device numbers: kept for the device that they were asked for, and not kept after a
failed query (compiled here as plain C++)."""

import os
import shutil
import subprocess

import pytest

from post_weight_quantization_03_gb300 import build_lib

PROGRAM = r"""
#include <cstdio>
#include "per_device.cuh"
int main() {
  static gptq::PerDevice<9> known;
  int asked = 0;
  auto gives = [&](int n) { return [&asked, n]() { ++asked; return n; }; };
  std::printf("%d ", known.get(0, 3, gives(46), 1));    // asked
  std::printf("%d ", known.get(0, 3, gives(99), 1));    // kept
  std::printf("%d ", known.get(1, 3, gives(40), 1));    // another device
  std::printf("%d ", known.get(0, 4, gives(30), 1));    // another key
  std::printf("%d ", known.get(1, 4, gives(0), 33));    // failed: the estimate, not kept
  std::printf("%d ", known.get(1, 4, gives(31), 33));
  std::printf("%d ", known.get(1, 4, gives(32), 33));
  std::printf("%d ", known.get(500, 4, gives(7), 33));  // past the table: asked each time
  std::printf("%d ", known.get(500, 4, gives(8), 33));
  std::printf("%d\n", asked);
}
"""


def test_numbers_belong_to_their_device(tmp_path):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("no g++")
    src, exe = tmp_path / "p.cpp", tmp_path / "p"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-x", "c++", "-I", build_lib.CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    assert out.split() == ["46", "46", "40", "30", "33", "31", "31", "7", "8", "7"]
    with open(os.path.join(build_lib.CSRC, "fp8_matmul.cu")) as f:
        text = f.read()
    assert "PerDevice" in text and "static std::atomic" not in text
