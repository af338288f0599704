"""Counts kept per device (csrc/per_device.h), as a program for the host: another device gets its own answer, each is
asked for once, and devices past the table are asked each time."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sampling_gated_lora_b200", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "per_device.h"
int main() {
  static uno::PerDevice<9> kept;
  int asked = 0;
  auto count = [&](int device, int slot) {
    return kept.get(device, slot, [&] { ++asked; return 100 * (device + 1) + slot; });
  };
  bool ok = count(0, 2) == 102 && count(1, 2) == 202 && count(1, 3) == 203 && asked == 3;
  ok = ok && count(0, 2) == 102 && count(1, 2) == 202 && asked == 3;
  ok = ok && count(64, 1) == 6501 && count(64, 1) == 6501 && count(-1, 1) == 1 && asked == 6;
  std::printf(ok ? "ok\n" : "wrong\n");
  return ok ? 0 : 1;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_each_device_has_its_own_counts(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout == "ok\n"
