"""What the feed-forward block's product kernel may read: a host program walks its tiles and
slices over small sizes with the functions the kernel uses (csrc/ffn_reads.hpp)."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "matrix_orthogonalising_optimizer_muon_amd", "csrc")

COMMON = r"""
#include <cstdio>
#include <initializer_list>
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

# K-contiguous operands: tiles of 32 to 256 rows (gate: half of each from Wg and Wu, over the hidden
# size rounded up to 64), 16-byte chunks at a lane offset and a scalar offset along the rows.
CONTIGUOUS = COMMON + r"""
int main() {
  long long walked = 0;
  const int kRows[] = {1, 2, 15, 16, 17, 31, 32, 33, 40, 63, 64, 65, 97, 129, 200, 257};
  for (int es = 2; es <= 4; es += 2)
    for (int K : {1, 3, 4, 7, 8, 9, 31, 32, 33, 63, 64, 65, 96, 127, 128, 129, 200})
      for (int R : kRows)
        for (int wide = 0; wide < 2; ++wide)
          for (int bm : {16, 32, 64, 128, 256})
            for (int padded = 0; padded < 2; ++padded) {
              const int bk = 128 / es;
              const long long ld = up(K, 16 / es) + wide * (16 / es);
              const long long end = up(((R - 1) * ld + K) * es, 16);
              const long long covered = padded ? up(R, 64) : R;
              for (int m0 = 0; m0 < covered; m0 += bm) {
                const int left = R - m0, bytes = ffn_bytes(least(left, bm), ld, K, es);
                const long long base = (long long)m0 * ld * es;
                for (int s = 0; s < up(K, bk) / bk + 7; ++s) {
                  const FfnWindow w = ffn_window(s * bk * es, ffn_end(bytes, K, es), bytes);
                  for (int row = 0; row < bm; ++row)
                    for (int c = 0; c < 8; ++c) {
                      const uint32_t lane = (uint32_t)((ffn_row(row, left) * ld + c * (16 / es)) * es);
                      ++walked;
                      const long long at = base + (long long)lane + w.at;
                      const bool sum = (long long)lane + w.at < w.bytes;          // lane + scalar against the bound
                      const bool difference = lane < (uint32_t)(w.bytes - w.at);  // lane against what is left
                      if ((sum || difference) && at + 16 > end) {
                        printf("es %d K %d rows %d ld %lld tile %d m0 %d slice %d row %d chunk %d: reads at %lld of %lld\n", es,
                               K, R, ld, bm, m0, s, row, c, at, end);
                        return 1;
                      }
                      const bool valid = row < left && s * bk + c * (16 / es) < K;
                      if (valid && (!sum || !difference || at != ((m0 + row) * ld + s * bk + c * (16 / es)) * es)) {
                        printf("es %d K %d rows %d m0 %d slice %d row %d chunk %d: a valid chunk is not read\n", es, K, R, m0,
                               s, row, c);
                        return 1;
                      }
                    }
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


def test_contiguous_operands_stay_inside(run):
    """Slices past the last one, one row left, tiles wholly in the padding: nothing behind the
    operand is read, however the hardware counts the scalar offset."""
    r = run("contiguous", CONTIGUOUS)
    assert r.returncode == 0 and "walked" in r.stdout, r.stdout
