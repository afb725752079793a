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
constexpr int32_t ffn_bytes(int32_t rows, int64_t ld, int64_t last, int es) {
  return rows > 0 && last > 0 ? static_cast<int32_t>((((rows - 1) * ld + last) * es + 15) & ~int64_t{15}) : 0;
}

}  // namespace muon
