"""Buffer offsets of the products' row operands, computed by the library's own
function in a program for the host."""

import os
import shutil
import subprocess

import pytest

from bit_quantized_moe_token_amd import build

PROGRAM = """
#include <cstdio>
#include "gemm.hpp"
using namespace moeq;

// Rows of `width` bytes, `stride` apart; the range ends with the last row.
// Stages 0 .. last + 8, as the longest ring moves them.  The range check is
// (lane offset) against (range - uniform offset), both unsigned.
int main() {
  long bad = 0, moved = 0;
  for (int width : {16, 32, 112, 128, 144, 256, 2000, 8192, 28672})
    for (int stride : {width, width + 16, 4 * width})
      for (int rows : {1, 2, 16, 256}) {
        const uint32_t range = (uint32_t)(rows - 1) * stride + width;
        for (int x : {0, rows / 2, rows - 1, -1})
          for (int t = 0; t < (width + kStageBytes - 1) / kStageBytes + 9; ++t)
            for (int piece = 0; piece < kStageBytes; piece += 16) {
              const StageOffsets o = stage_offsets(t, piece, width, x < 0 ? kNowhere : (uint32_t)x * stride + piece);
              const bool there = x >= 0 && t * kStageBytes + piece < width;
              bool ok = o.soff <= range && there == (o.voff < range - o.soff);
              if (there) {
                ok = ok && o.voff + o.soff == (uint32_t)x * stride + t * kStageBytes + piece && o.voff + o.soff + 16 <= range;
                ++moved;
              }
              bad += !ok;
            }
      }
  std::printf("%ld %ld\\n", bad, moved);
}
"""


@pytest.mark.skipif(not os.path.exists(build.HIPCC) and not shutil.which(build.HIPCC), reason="no compiler")
def test_offsets_stay_within_the_range(tmp_path):
    src, exe = tmp_path / "offsets.hip", tmp_path / "offsets"
    src.write_text(PROGRAM)
    cmd = [build.HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O1", "-Wno-everything", "-I", build.CSRC,
           str(src), "-o", str(exe)]
    subprocess.run(cmd, check=True, capture_output=True, timeout=300)
    bad, moved = map(int, subprocess.run([str(exe)], check=True, capture_output=True, timeout=60).stdout.split())
    assert moved > 0 and bad == 0
