// What the product kernel of the feed-forward block (ffn.hip) may read of an operand, as plain
// constexpr functions: the kernel and a host program that walks every tile and slice use the
// same ones.
#pragma once

#include <cstdint>

namespace muon {

// Buffer bound, in bytes from the first element of a tile's piece of an operand: `rows` rows
// `ld` elements apart, of which the last one has `last` elements left. Rounded up to whole
// 16-byte chunks: rows are 16-byte aligned, so such a chunk shares its page with a valid
// element. Nothing is left (0: every access is out of bounds) without rows, and for a tile that
// starts behind the row's last element: there the size would come out negative and, read as
// unsigned, bound nothing.
// (One select: a branch here would cut the product loop in two.)
constexpr int32_t ffn_bytes(int32_t rows, int64_t ld, int32_t last, int es) {
  const int32_t bytes = static_cast<int32_t>(((rows - 1) * ld + last) * es + 15) & ~15;
  return (rows < last ? rows : last) > 0 ? bytes : 0;
}

// Row of a K-contiguous operand's tile that a lane reads: rows behind the last repeat it, and a
// tile without rows (gate: wholly in the padding of the hidden size) names its first.
constexpr int32_t ffn_row(int32_t row, int32_t rows) {
  return row < rows ? row : (rows > 0 ? rows - 1 : 0);
}

// A slice of a K-contiguous operand: the bound and the scalar offset `at` (bytes along the rows)
// of its loads. The ring asks for slices past the last one, at >= `end` (the rows' valid bytes; 0
// for a tile without rows); those get an empty bound at offset 0 and read zeros. So the offset
// never exceeds the bound, whether the hardware checks lane offset + scalar offset against it, or
// the lane offset against the difference (which would wrap).
struct FfnWindow {
  int32_t bytes, at;
};
constexpr int32_t ffn_end(int32_t bytes, int32_t K, int es) {
  return bytes > 0 ? K * es : 0;
}
constexpr FfnWindow ffn_window(int32_t at, int32_t end, int32_t bytes) {
  return at < end ? FfnWindow{bytes, at} : FfnWindow{0, 0};
}

}  // namespace muon
