"""Which rows the tiles of the tensor-core attention over the 4-bit cache take:
the kernel's own arithmetic, compiled for the host."""
import ctypes
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_tree_bit_gb300",
                    "csrc")
SOURCE = r"""
#include <stdint.h>
#include "kv4_rows.cuh"
using namespace sdv;

// Every lane's row of every segment of m nodes and G query heads a kv head: a
// row outside [0, G m) would read past the slopes of the last kv head.  Each
// row has to be some lane's.  Returns -1, or what failed.
template <bool WIDE>
static int check(int G, int m) {
  const int gm = G * m, nc = (gm + 255) / 256;
  static uint8_t seen[1024];
  for (int i = 0; i < gm; i++) seen[i] = 0;
  for (int rc = 0; rc < nc; rc++) {
    const TcRowsOf<WIDE> w(gm, nc, rc);
    if (w.rows < 1 || w.rows > 256 || w.of(0) > 128 || w.of(1) > 128) return 1000;
    if (!WIDE && w.rows * w.copies > 128) return 1001;
    for (int t = 0; t < 2; t++)
      for (int lane = 0; lane < 128; lane++) {
        const int ridx = lane % (128 / w.copies), row = w.row(t, ridx);
        if (row < 0 || row >= gm) return row;
        if (ridx < w.of(t)) seen[row] = 1;
      }
  }
  for (int i = 0; i < gm; i++)
    if (!seen[i]) return 1002;
  return -1;
}

extern "C" int rows_check(int wide, int G, int m) { return wide ? check<true>(G, m) : check<false>(G, m); }
"""


@pytest.fixture(scope="module")
def check(tmp_path_factory):
    d = tmp_path_factory.mktemp("rows")
    src, so = d / "rows.cpp", d / "rows.so"
    src.write_text(SOURCE)
    cxx = shutil.which("g++") or shutil.which("c++")
    assert cxx
    subprocess.run([cxx, "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(so)], check=True)
    return ctypes.CDLL(str(so)).rows_check


def test_no_lane_takes_a_row_past_the_request(check):
    """A call whose largest request has more than 128 rows a kv head takes
    every request on the wide form, the smallest ones too."""
    for G in range(1, 17):
        for m in range(1, 65):
            assert check(1, G, m) == -1, (G, m)
            if G * m <= 128:
                assert check(0, G, m) == -1, (G, m)
