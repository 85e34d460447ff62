"""Numbers that the host asks for once on each device, compiled without CUDA."""
import re
import shutil
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parents[1] / "block_diffusion_speculative_02_gb300" / "csrc"

PROGRAM = """
#include "per_device.h"
#include <cstdio>
int main() {
  static dflash::PerDevice kept;
  int asked = 0, give = 0;
  const auto ask = [&] { ++asked; return give; };
  if (kept.get(0, ask) != 0 || kept.get(0, ask) != 0 || asked != 2) return 1;   // failed: again
  give = 152;
  if (kept.get(0, ask) != 152 || asked != 3) return 2;
  give = 76;
  if (kept.get(0, ask) != 152 || asked != 3) return 3;                          // kept
  if (kept.get(1, ask) != 76 || kept.get(1, ask) != 76 || asked != 4) return 4; // its own
  if (kept.get(0, ask) != 152 || kept.get(63, ask) != 76 || asked != 5) return 5;
  if (kept.get(64, ask) != 76 || kept.get(64, ask) != 76 || kept.get(-1, ask) != 76) return 6;
  return asked == 8 ? 0 : 7;
}
"""


def test_kept_for_each_device_and_only_what_did_not_fail(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no C++ compiler")
    src = tmp_path / "kept.cpp"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-Wall", "-I", str(CSRC), str(src), "-o",
                    str(tmp_path / "kept")], check=True)
    assert subprocess.run([str(tmp_path / "kept")]).returncode == 0


def test_products_keep_no_answer_of_a_device_for_the_process():
    """(A static filled from whichever device calls first; constants apart.)"""
    for path in sorted(CSRC.glob("fp8*")):
        assert not re.search(r"static const (int|bool|long long) \w+ = ", path.read_text()), path.name
