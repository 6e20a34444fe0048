"""The slices of a batch over the launches of a one-token step
(csrc/row_slices.hpp), on the host: every row once, in order, up to the largest
batch of the C ABI."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "selective_state_space_28_amd", "csrc")

MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include "row_slices.hpp"
int main(int argc, char** argv) {
  for (int k = 1; k < argc; ++k) {
    const int batch = std::atoi(argv[k]);
    long long next = 0, calls = 0;
    const int rc = ssm::by_row_slices(batch, 0, [&](int b0, int rows) {
      ++calls;
      if (b0 != next || rows < 1 || rows > ssm::kMaxGridRows) return 1;
      next += rows;
      return 0;
    });
    std::printf("%d %lld %lld\n", rc, next, calls);
  }
  long long seen = 0;  // a failing launch ends them
  const int rc = ssm::by_row_slices(200000, 0, [&](int, int) { return ++seen == 2 ? 7 : 0; });
  std::printf("%d %lld\n", rc, seen);
}
"""


def test_every_row_once(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ is not available")
    src, exe = tmp_path / "slices.cpp", str(tmp_path / "slices")
    src.write_text(MAIN)
    # -ftrapv: signed overflow ends the program
    subprocess.run([gxx, "-std=c++17", "-O1", "-ftrapv", "-I", CSRC, "-o", exe, str(src)], check=True)
    top = 2**31 - 1
    batches = [0, 1, 65534, 65535, 65536, 131070, 131071, 32768 * 65535, 32768 * 65535 + 1, top - 1, top]
    out = subprocess.run([exe, *map(str, batches)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stderr
    rows = [tuple(map(int, line.split())) for line in out.stdout.splitlines()]
    assert rows == [(0, b, -(-b // 65535)) for b in batches] + [(7, 2)]
