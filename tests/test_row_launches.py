"""The rows of one launch of a row kernel (layer norm, rows to 8 bits): whole workgroups,
so that no row belongs to two launches, as many as 2^32 work-items allow."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "convolution_forward_amd", "csrc")

DRIVER = """
#include <stdio.h>
#include "rows_plan.h"
int main() {
  using convfwd::rows_of_launch;
  const int64_t limit = 1LL << 32;
  for (int64_t items = 1; items <= 131072; items = items < 600 ? items + 1 : items * 2 - 7)
    for (int64_t teams = 1; teams <= 64; ++teams) {
      const int64_t rows = rows_of_launch(items, teams);
      const bool whole = rows > 0 && rows % teams == 0;
      const bool fits = rows * items < limit, full = (rows + teams) * items > limit - limit / 128;
      if (!whole || !fits || !full) {
        printf("%lld rows of %lld work-items, %lld a workgroup\\n", (long long)rows,
               (long long)items, (long long)teams);
        return 1;
      }
    }
  return 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_whole_workgroups(tmp_path):
    src, exe = tmp_path / "driver.cpp", str(tmp_path / "driver")
    src.write_text(DRIVER)
    subprocess.run(["g++", "-std=c++17", "-I", os.path.join(ROOT, "include"), "-I", CSRC, str(src),
                    "-o", exe], check=True, capture_output=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout
