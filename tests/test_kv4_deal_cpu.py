"""How the kernel for prefixes of many rows deals its rows, compiled and run on the host: up to the rows that a call
takes, every strip of 32 rows belongs to exactly one tile of at most 8 or 4 strips."""
import os
import subprocess

import quantized_matmul_quantize_amd as qmm

SOURCE = r"""
#include <cstdint>
#include <cstdio>
#include <initializer_list>

#include "kv4_deal.h"

int check(int strips, int most) {
  const int tiles = (strips + most - 1) / most;
  int next = 0;
  for (int tile = 0; tile < tiles; ++tile) {
    const int first = qmm::first_strip(tile, strips, tiles), end = qmm::first_strip(tile + 1, strips, tiles);
    const int64_t even = strips / tiles;
    if (first != next || end - first < even || end - first > even + 1 || end - first > most || first < 0) {
      std::printf("%d strips in %d tiles: tile %d from %d to %d\n", strips, tiles, tile, first, end);
      return 1;
    }
    next = end;
  }
  if (next != strips) std::printf("%d strips: %d dealt\n", strips, next);
  return next != strips;
}

int main() {
  for (int most : {8, 4}) {
    for (int strips = 1; strips < 2000; ++strips)
      if (check(strips, most)) return 1;
    // 2^22 rows and around them; up to 2^31 - 1
    for (int strips : {92681, 92683, 131071, 131072, 131073, 262143, 262144, 262145, 1 << 20, 5000011, (1 << 26) - 1, 1 << 26})
      if (check(strips, most)) return 1;
  }
  return 0;
}
"""


def test_every_strip_of_rows_is_in_one_tile(tmp_path):
    (tmp_path / "deal.cpp").write_text(SOURCE)
    csrc = os.path.join(os.path.dirname(qmm.__file__), "csrc")
    subprocess.check_call(["g++", "-std=c++17", "-O1", "-ftrapv", "-I", csrc, "-o", str(tmp_path / "deal"), str(tmp_path / "deal.cpp")])
    done = subprocess.run([str(tmp_path / "deal")], stdout=subprocess.PIPE, text=True)
    assert done.returncode == 0, done.stdout
