"""The row kernels' index arithmetic (csrc/ia_rows.h), compiled for the host and checked for every row length."""
import os
import subprocess

from ssm_token_mixer_b200 import build

PROGRAM = r"""
#include "ia_rows.h"
#include <cstdio>
// Every vector that a thread of a group fetches for a row, past the row's end too: its source is aligned to 16 bytes and
// inside the tensor, and what it copies ends with the row.
int main() {
  for (int size = 2; size <= 4; size += 2) {
    const int V = 16 / size, rows = 2 * V + 1;
    for (int D = 1; D <= 700; ++D)
      for (long long row = 0; row < rows; ++row) {
        const long long first = row * D;
        const int mis = static_cast<int>(first % V);
        for (int c = -mis; c < 2 * D + 64; c += V) {
          const long long from = first + ia::copy_column(c, D, mis);
          const int bytes = ia::copy_bytes(c, D, size);
          const bool ok = from % V == 0 && from >= 0 && from * size + bytes <= (first + D) * size &&
                          bytes == (c >= D ? 0 : D - c < V ? (D - c) * size : 16) && (bytes == 0 || from == first + c);
          if (!ok) {
            std::printf("size %d D %d row %lld c %d: from %lld, %d bytes\n", size, D, row, c, from, bytes);
            return 1;
          }
        }
      }
  }
  return 0;
}
"""


def test_copies_start_on_a_boundary_inside_the_tensor(tmp_path):
    src, exe = tmp_path / "rows.cpp", str(tmp_path / "rows")
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", os.path.join(build.CSRC), str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
