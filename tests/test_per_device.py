"""The set-up of a kernel on each device (csrc/exq_per_device.h), on the CPU: once where it worked, again where it failed."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_weight_exq_gb300", "csrc")

PROGRAM = """
#include "exq_per_device.h"
#include <cstdio>
int main() {
  static exq::PerDevice state;
  int calls[2] = {0, 0}, fail = 1;
  const auto on = [&](int d) { return state.once(d, [&] { ++calls[d]; return true; }); };
  bool ok = on(0) && on(0) && calls[0] == 1;                                   // once on a device
  ok = ok && on(1) && calls[1] == 1 && on(1) && on(0) && calls[1] == 1 && calls[0] == 1;   // and on the next one too
  int tries = 0;
  const auto flaky = [&] { ++tries; return fail-- <= 0; };
  ok = ok && !state.once(2, flaky) && state.once(2, flaky) && state.once(2, flaky) && tries == 2;
  ok = ok && !state.once(-1, [] { return true; }) && !state.once(64, [] { return true; });
  std::puts(ok ? "ok" : "wrong");
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_set_up_is_per_device(tmp_path):
    src = tmp_path / "t.cpp"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(tmp_path / "t"), "-pthread"], check=True)
    assert subprocess.run([str(tmp_path / "t")], capture_output=True, text=True, check=True).stdout.strip() == "ok"


def test_no_kernel_attribute_is_set_once_a_process():
    # cudaFuncSetAttribute reaches the current device only
    for name in os.listdir(CSRC):
        text = open(os.path.join(CSRC, name)).read()
        for call in re.finditer(r"call_once", text):
            assert "cudaFuncSetAttribute" not in text[call.start():call.start() + 400], name
