"""Host-side test of what fa_decode_join_kernel reads and writes by way of the workspace's
entries (csrc/fa_decode.cuh): a decode kernel that gave up leaves them as they were, so any
words may be there."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "io_aware_exact_23_b200", "csrc")

# Entries of random words, of words near each limit, and every entry that a call can write: the slots
# that are read (row 2c + 1, then 2 (c + i)) and the output rows, for the blocks of a grid that pass.
MAIN = r"""
#include <cstdio>
#include <cstdint>
#include "fa_decode.cuh"
static uint64_t state = 88172645463325252ull;
static int word() {
  state ^= state << 13; state ^= state >> 7; state ^= state << 17;
  const int near[] = {-2147483647 - 1, -1, 0, 1, 2, 3, 7, 8, 9, 159, 160, 295, 296, 319, 320, 321, 640, 2147483647};
  const int r = static_cast<int>(state >> 16);
  return (r & 3) ? near[static_cast<unsigned>(r >> 4) % (sizeof(near) / sizeof(near[0]))] : r;
}
int main() {
  const int shapes[][3] = {{1, 1, 1}, {3, 8, 4}, {2, 66, 33}, {5, 40, 40}, {300, 2, 1}};  // B, Hq, G
  long passed = 0;
  for (const auto &s : shapes) {
    const int B = s[0], Hq = s[1], G = s[2];
    for (long t = 0; t < 3000000; ++t) {
      const int b = word(), row = word(), parts = word(), c = word();
      if (!fa::decode_entry_ok(b, row, parts, c, B, Hq)) continue;
      ++passed;
      const int64_t last = parts > 1 ? 2 * (int64_t(c) + parts - 1) : 0, first = 2 * int64_t(c) + 1;
      if (first < 0 || first >= 2 * fa::kDecodeMaxCtas || last >= 2 * fa::kDecodeMaxCtas) return 1;
      for (int g = 0; g < 32 && row % G + g < G; ++g)
        if (int64_t(b) * Hq + row + g >= int64_t(B) * Hq || row + g >= Hq) return 2;
    }
    // What decode_note writes passes, an entry of no parts does not.
    for (int b = 0; b < B; ++b)
      for (int row = 0; row < Hq; ++row)
        for (int c = 0; c < fa::kDecodeMaxCtas; c += 37) {
          if (!fa::decode_entry_ok(b, row, fa::kDecodeMaxCtas - c, c, B, Hq)) return 3;
          if (!fa::decode_entry_ok(b, row, 1, c, B, Hq)) return 3;
          if (fa::decode_entry_ok(b, row, 0, c, B, Hq)) return 4;
        }
  }
  std::printf("%ld\n", passed);
  return passed > 1000 ? 0 : 5;
}
"""


def test_no_entry_leads_out_of_the_buffers(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src, exe = tmp_path / "entries.cu", tmp_path / "entries"
    src.write_text(MAIN)
    subprocess.check_call([nvcc, "-std=c++17", "-gencode", "arch=compute_100a,code=sm_100a", "-I", CSRC, "-o", str(exe), str(src)])
    got = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert got.returncode == 0, (got.returncode, got.stdout)


def test_the_join_kernel_checks_before_it_follows():
    """The check stands between the entry's load and its first use."""
    src = open(os.path.join(CSRC, "fa_decode.cuh")).read()
    body = src[src.index("fa_decode_join_kernel(const"):]
    load, check, use = body.index("p.meta[blockIdx.x]"), body.index("decode_entry_ok("), body.index("auto row")
    assert load < check < use
