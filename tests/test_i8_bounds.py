"""The int8 products' operand reads stay inside their matrices: every offset
that a lane can form (tenant_composite_lora_amd/csrc/i8_index.hpp, compiled
for the host), for rows of every length around a block, rows and blocks past
the end among them."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "tenant_composite_lora_amd", "csrc")
ROCM_INCLUDE = "/opt/rocm/include"

DRIVER = r"""
#include <cstdio>
#include "i8_index.hpp"
using namespace tcl;
int main() {
  long bad = 0, seen = 0;
  for (int K = 16; K <= 272; K += 16)
    for (int n = 1; n <= 40; n += n < 3 ? 1 : 6)
      for (int kind = 0; kind < 3; ++kind) {
        const int kb = (K + 63) / 64;
        const Mat8 m{nullptr, kind == 1 ? K + 48 : K, n, K / 16, kb, kind == 2};
        // rows end where the last one does: nothing behind it belongs to them
        const long size = kind == 2 ? (n + 15) / 16 * kb * 1024L : (n - 1) * m.ld + K;
        for (int r = 0; r < 300; ++r)
          for (int b = 0; b < kb + 40; ++b)
            for (int g = 0; g < 4; ++g) {
              const long at = mat_at(m, r, g) + long(block_or_first(K, b, g)) * mat_step(m);
              ++seen;
              if (at < 0 || at + 16 > size || at % 16) {
                if (!bad++) std::printf("K %d rows %d kind %d: row %d block %d chunk %d reads at %ld of %ld\n",
                                        K, n, kind, r, b, g, at, size);
              }
              // what lies in the row is read from its own place
              if (chunk_in(K, b, g) && r < n && kind < 2 && at != r * m.ld + 64 * b + 16 * g) ++bad;
            }
      }
  std::printf("%ld reads, %ld bad\n", seen, bad);
  return bad != 0;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None or not os.path.isdir(ROCM_INCLUDE),
                    reason="needs g++ and the ROCm headers")
def test_every_operand_read_lies_in_its_matrix(tmp_path):
    src, exe = tmp_path / "bounds.cpp", tmp_path / "bounds"
    src.write_text(DRIVER)
    b = subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", ROCM_INCLUDE,
                        "-I", CSRC, str(src), "-o", str(exe)], capture_output=True, text=True)
    assert b.returncode == 0, b.stderr[-3000:]
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
