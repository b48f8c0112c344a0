"""The set-up that a launch does once on every device: a failure is not remembered, a device does not stand for another
(CPU; a host program compiled on the spot)."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "routing_quant_expert_amd", "csrc")
PROGRAM = r"""
#include "moe_once.h"
#include <cstdio>
enum Error { kOk = 0, kBad = 7 };
static int calls = 0;
static Error answer = kOk;
static Error set_up() { ++calls; return answer; }
#define CHECK(c) do { if (!(c)) { printf("line %d: %s\n", __LINE__, #c); return 1; } } while (0)
int main() {
  static moe::OncePerDevice once;
  answer = kBad;
  CHECK(once(0, set_up) == kBad && calls == 1);
  CHECK(once(0, set_up) == kBad && calls == 2);    // tried again
  answer = kOk;
  CHECK(once(0, set_up) == kOk && calls == 3);
  CHECK(once(0, set_up) == kOk && calls == 3);     // there
  CHECK(once(1, set_up) == kOk && calls == 4);     // another device
  CHECK(once(63, set_up) == kOk && calls == 5);
  CHECK(once(63, set_up) == kOk && calls == 5);
  CHECK(once(64, set_up) == kOk && once(64, set_up) == kOk && calls == 7);   // past the bits: every time
  CHECK(once(0, set_up) == kOk && calls == 7);
  return 0;
}
"""


def test_once_per_device(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True, timeout=60)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=20)
    assert r.returncode == 0, r.stdout
