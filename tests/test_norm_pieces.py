"""The layer norm's copies of rows of any alignment read nothing outside their
array, and all of their row: the address arithmetic of the kernel's copies
over small and odd shapes, compiled for the host."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kronecker_factored_gptq_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "rows_copy.h"
using namespace bakron;

// One array of T rows of d elements of es bytes that begins `base` bytes into
// an aligned piece; a thread block of `warps` warps, NV vectors a lane.
static int check(int T, int d, int es, int base, int nv, int warps) {
  const long lo = base, hi = base + (long)T * d * es;
  for (int row = 0; row < T; ++row) {
    const long begin = base + (long)row * d * es;
    std::vector<char> got(d * es, 0);
    for (int w = 0; w < warps; ++w) {
      const int c0 = w * 32 * nv * (16 / es);
      const int shift = (int)(begin & 15);
      const long first = begin + (long)c0 * es - shift;      // the warp's first piece
      const int left = (d - c0) * es + shift;
      const long front = ((long)row * d + c0) * es;
      const int before = front < 16 ? (int)front : 16;
      if (left <= 0 || c0 >= d) continue;
      for (int lane = 0; lane < 32; ++lane)
        for (int i = 0; i <= nv; ++i) {
          if (i == nv && lane > 0) break;
          const int at = lane * 16 + i * 512;
          const PieceBytes p = piece_bytes(before, shift, left, at);
          for (int b = p.from; b < p.to; ++b) {
            const long a = first + at + b;
            if (a < lo || a >= hi) {
              std::printf("T %d d %d es %d base %d row %d: byte %ld outside [%ld, %ld)\n", T, d, es, base, row, a, lo, hi);
              return 1;
            }
            if (a >= begin && a < begin + (long)d * es) got[a - begin] = 1;
          }
        }
    }
    for (char g : got)
      if (!g) {
        std::printf("T %d d %d es %d base %d row %d: a byte of the row is not read\n", T, d, es, base, row);
        return 1;
      }
  }
  return 0;
}

int main() {
  const int ds[] = {1, 2, 3, 4, 5, 6, 7, 8, 9, 15, 16, 17, 31, 33, 127, 255, 1023, 1025, 2049, 4100};
  for (int es = 2; es <= 4; es += 2)
    for (int d : ds)
      for (int base = 0; base < 16; base += es)
        for (int T = 1; T <= 20; T += 1 + T / 4)
          for (int nv = 1; nv <= 8; nv *= 2) {
            const int columns = 32 * nv * (16 / es);
            if (check(T, d, es, base, nv, (d + columns - 1) / columns)) return 1;
          }
  return 0;
}
"""


def test_copies_stay_inside_their_array(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "pieces.cpp", tmp_path / "pieces"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-O2", "-I", CSRC, "-o", str(exe), str(src)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
