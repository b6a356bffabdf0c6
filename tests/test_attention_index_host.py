"""The attention tiles' index arithmetic, checked thread by thread on the host
(no GPU): a whole tile's loads stay within their rows' heads, fill the tile's
columns, and the tile's places are each used once."""
import shutil
import subprocess

import pytest

from padding_free_pair_amd.build import CSRC

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "nt_attention_index.hpp"

template <int SIZE, int ROWS, int DP, int THREADS> void check() {
  typedef nt::AtLoadMap<SIZE, ROWS, DP, THREADS> M;
  typedef typename M::L L;
  for (long ld : {(long)DP, (long)DP * 3 + 8, 1L << 22}) {
    std::vector<int> filled(ROWS * L::chunks, 0);
    for (int u = 0; u < M::pieces; ++u)
      for (int t = 0; t < THREADS; ++t) {
        const long at = M::whole(t, u, (uint32_t)ld) / SIZE;
        const int row = M::row(t, u), col = M::col(t, u);
        // a load of 16 bytes within its row's head, the last one of the array among them
        if (row < 0 || row >= ROWS || at < row * ld || at + L::vec > row * ld + DP) {
          std::printf("SIZE %d ROWS %d DP %d ld %ld thread %d piece %d: row %d, elements %ld ..\n",
                      SIZE, ROWS, DP, ld, t, u, row, at - row * ld);
          std::exit(1);
        }
        // the chunk that its place in LDS stands for
        const int place = t + u * THREADS;
        if (L::at(row, col) != place * L::vec || (col < DP && at != row * ld + col)) {
          std::printf("SIZE %d ROWS %d DP %d: thread %d piece %d misplaced\n", SIZE, ROWS, DP, t, u);
          std::exit(2);
        }
        if (col < DP) filled[row * L::chunks + col / L::vec] += 1;
      }
    for (int r = 0; r < ROWS; ++r)
      for (int c = 0; c < DP; c += L::vec)
        if (filled[r * L::chunks + c / L::vec] != 1) std::exit(3);
  }
  std::vector<int> used(ROWS * L::pitch, 0);
  for (int r = 0; r < ROWS; ++r)
    for (int c = 0; c < DP; ++c) {
      const int at = L::at(r, c);
      if (at < 0 || at >= ROWS * L::pitch || used[at]++) std::exit(4);
    }
}
template <int SIZE, int DP> void widths() {
  check<SIZE, 64, DP, 256>();
  check<SIZE, 128, DP, 256>();
  check<SIZE, 64, DP, 128>();
}
int main() {
  widths<2, 32>(); widths<2, 64>(); widths<2, 96>(); widths<2, 128>();
  widths<4, 32>(); widths<4, 64>(); widths<4, 96>(); widths<4, 128>();
  return 0;
}
"""


def test_whole_tiles_stay_within_their_rows(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("needs g++")
    src, exe = tmp_path / "index.cpp", tmp_path / "index"
    src.write_text(PROGRAM)
    made = subprocess.run([gxx, "-std=c++17", "-O1", f"-I{CSRC}", str(src), "-o", str(exe)],
                          capture_output=True, text=True)
    assert made.returncode == 0, made.stderr
    ran = subprocess.run([str(exe)], capture_output=True, text=True)
    assert ran.returncode == 0, (ran.returncode, ran.stdout)
