"""Set-up of kernels that CUDA keeps per device: done once on every device, and
again after a failure (no GPU: the bookkeeping alone, with made-up devices)."""
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "flashattention_attn_fwd_gb300", "csrc")

PROGRAM = r"""
#include <cassert>
#include <thread>
#include <vector>
#include "per_device.h"

enum Error { kOk = 0, kBad = 7 };
static fl::OncePerDevice once;

int main() {
  int calls[3] = {0, 0, 0};
  auto good = [&](int dev) { return once.run(dev, [&] { ++calls[dev]; return kOk; }); };
  assert(good(0) == kOk && good(0) == kOk && calls[0] == 1);
  assert(calls[1] == 0 && good(1) == kOk && good(1) == kOk && calls[1] == 1);   // a second device
  int tries = 0;
  auto flaky = [&] { return ++tries == 1 ? kBad : kOk; };
  assert(once.run(2, flaky) == kBad);                                           // not kept
  assert(once.run(2, flaky) == kOk && once.run(2, flaky) == kOk && tries == 2);
  // what a step leaves is there for whoever finds it done
  static fl::OncePerDevice shared;
  static int value[4];
  std::vector<std::thread> all;
  int steps = 0, wrong[8] = {};
  for (int t = 0; t < 8; ++t)
    all.emplace_back([&, t] {
      for (int dev = 0; dev < 4; ++dev) {
        shared.run(dev, [&] { ++steps; value[dev] = 10 + dev; return kOk; });
        wrong[t] += value[dev] != 10 + dev;
      }
    });
  for (auto& t : all) t.join();
  for (int w : wrong) assert(w == 0);
  assert(steps == 4);
  return 0;
}
"""


def test_a_step_runs_once_on_every_device(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "once.cpp", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    subprocess.run([str(exe)], check=True, timeout=60)


def test_kernel_attributes_are_set_on_the_device_of_the_call():
    """Every limit that a launcher raises goes through the bookkeeping above: none
    is kept in a variable that the first device settles for all."""
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith((".cu", ".cuh", ".h")):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        uses = len(re.findall(r"\bcudaFuncSetAttribute\s*\(", text))
        assert uses == 0 or len(re.findall(r"\bon_this_device\s*\(", text)) >= uses, name
        assert not re.search(r"static const (cudaError_t|int) \w+ = (\[|cuda)", text), name
