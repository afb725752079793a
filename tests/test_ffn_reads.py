"""What the feed-forward block's product kernel may read: a host program walks its tiles and
slices over small sizes with the functions the kernel uses (csrc/ffn_reads.hpp)."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_orthogonalising_optimizer_muon_amd", "csrc")

COMMON = r"""
#include <cstdio>
#include <cstdint>
#include "ffn_reads.hpp"
using namespace muon;
static long long up(long long x, long long a) { return (x + a - 1) / a * a; }
static const int kTileN[] = {32, 64, 128, 256};
static int least(long long a, long long b) { return (int)(a < b ? a : b); }
"""

# Every stage's K-strided operand: K rows of N elements, tiles over the columns rounded up to 64
# (dgate writes the padding of dg, du and h too), slices of 128 bytes a row.
STRIDED = COMMON + r"""
int main() {
  long long walked = 0;
  for (int es = 2; es <= 4; es += 2)
    for (int K = 1; K <= 130; ++K)
      for (int N = 1; N <= 260; ++N)
        for (int wide = 0; wide < 2; ++wide)
          for (int bn : kTileN) {
            const int bk = 128 / es;
            const long long ld = up(N, 16 / es) + wide * (16 / es);
            const long long end = up(((K - 1) * ld + N) * es, 16);   // of the operand, whole chunks
            for (int n0 = 0; n0 < up(N, 64); n0 += bn)
              for (int k0 = 0; k0 < up(K, bk) + 7 * bk; k0 += bk) {  // up to 7 slices past the last
                const long long bytes = ffn_bytes(least(K - k0, bk), ld, N - n0, es);
                const long long base = (k0 * ld + n0) * es;
                ++walked;
                if (bytes < 0 || bytes % 16 != 0 || (bytes > 0 && base + bytes > end)) {
                  printf("es %d K %d N %d ld %lld tile %d n0 %d k0 %d: %lld bytes at %lld of %lld\n", es, K, N, ld, bn,
                         n0, k0, bytes, base, end);
                  return 1;
                }
                // what the tile needs: every valid element
                const int rows = least(K - k0, bk), cols = least(N - n0, bn);
                if (rows > 0 && cols > 0 && bytes < ((rows - 1) * ld + cols) * es) {
                  printf("es %d K %d N %d: valid elements cut off\n", es, K, N);
                  return 1;
                }
              }
          }
  printf("walked %lld\n", walked);
  return 0;
}
"""


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    def go(name, source):
        d = tmp_path_factory.mktemp(name)
        (d / "walk.cpp").write_text(source)
        subprocess.run(["g++", "-std=c++17", "-O2", "-I", CSRC, str(d / "walk.cpp"), "-o", str(d / "walk")], check=True)
        return subprocess.run([str(d / "walk")], capture_output=True, text=True, timeout=300)
    return go


def test_strided_operands_stay_inside(run):
    """A tile that starts behind the last column and a slice of one row left: no negative bound."""
    r = run("strided", STRIDED)
    assert r.returncode == 0 and "walked" in r.stdout, r.stdout
