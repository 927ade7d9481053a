"""How many parts a unit of the paged attention has, compiled for the host: the estimate that chooses the
join against the split itself."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

HARNESS = r"""
#include <cstdio>
#include <initializer_list>
#include "page_index.h"
using namespace mikv;
#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)
int main() {
  CHECK(parts_of_unit(5, 8, 160) == 5);   // 77 slots of 8 key heads: five tiles, whatever the warps
  CHECK(parts_of_unit(1, 8, 32) == 1);
  CHECK(parts_of_unit(4096, 1, 1216) == 1216 && parts_of_unit(512, 512, 1216) == 2);
  for (int64_t tiles : {1, 2, 5, 16, 17, 63, 512, 4096})
    for (int64_t units : {1, 3, 8, 24, 192, 1300})
      for (int64_t warps : {4, 20, 160, 608, 1216}) {
        const int64_t total = tiles * units, about = parts_of_unit(tiles, units, warps);
        const int workers = (int)(total < warps ? total : warps);
        for (int64_t u = 0; u < units; ++u) {
          const int parts = split_owner(total, workers, (u + 1) * tiles - 1) - split_owner(total, workers, u * tiles) + 1;
          CHECK(parts >= about && parts <= about + 2 && parts <= tiles);
        }
      }
  return 0;
}
"""


def test_parts_of_a_unit(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no g++")
    src = tmp_path / "parts.cpp"
    src.write_text(HARNESS)
    inc = os.path.join(ROOT, "mixed_precision_kv_balancer_gb300", "csrc")
    subprocess.run([gxx, "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", inc, str(src),
                    "-o", str(tmp_path / "parts")], check=True)
    res = subprocess.run([str(tmp_path / "parts")], capture_output=True, text=True)
    assert res.returncode == 0, res.stdout + res.stderr
