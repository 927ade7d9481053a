"""Index arithmetic of the choice of blocks, compiled for the host: where bounds lie in shared memory."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

HARNESS = r"""
#include <vector>
#include "block_index.h"
using namespace mikv;
int main() {
  for (uint32_t base = 0; base < 512; base += 16) {   // the buffer may begin at any 16 bytes
    std::vector<int> memory(base + 32 * kBoundBytes, -1);
    for (uint32_t e = 0; e < 32; ++e)
      for (uint32_t piece = 0; piece < 16; ++piece) {
        const uint32_t at = base + bound_at(e, piece);
        if (at % 16 || at >= memory.size() || memory[at] != -1) return 1;
        memory[at] = e * 16 + piece;
      }
    for (uint32_t g = 0; g < 8; ++g)
      for (uint32_t t = 0; t < 4; ++t)
        for (uint32_t j = 0; j < 4; ++j)
          for (uint32_t k = 0; k < 4; ++k)
            if (memory[base + bound_of_lane(bound_at(g, t), j, k)] != (int)((8 * j + g) * 16 + 4 * k + t)) return 2;
  }
  // eight lanes of a read, two blocks beside one another, meet all banks once
  for (uint32_t g = 0; g < 8; g += 2)
    for (uint32_t k = 0; k < 4; ++k) {
      unsigned banks = 0;
      for (uint32_t l = 0; l < 8; ++l) banks |= 1u << bound_of_lane(bound_at(g + l / 4, l % 4), 0, k) / 16 % 8;
      if (banks != 255) return 3;
    }
  return 0;
}
"""


def test_bounds_are_read_where_they_were_written(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "block_index.cpp"
    src.write_text(HARNESS)
    inc = os.path.join(ROOT, "mixed_precision_kv_balancer_gb300", "csrc")
    subprocess.run([gxx, "-O1", "-std=c++17", "-fsanitize=undefined,address", "-fno-sanitize-recover", "-I", inc, str(src),
                    "-o", str(tmp_path / "block_index")], check=True)
    res = subprocess.run([str(tmp_path / "block_index")], capture_output=True, text=True)
    assert res.returncode == 0, res.returncode

