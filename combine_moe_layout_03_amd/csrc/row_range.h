// Rows of a tile that starts at row `row0` of an expert whose rows end before
// `row_end` (row0 < row_end).  A tile's last rows may pass the expert's end,
// and row0 + r the largest int32, so both questions are asked of differences.
// Host arithmetic only, without HIP, so that a CPU test can compile it.
#pragma once

#include <stdint.h>

namespace moe {

// Whether the tile's row r (0 <= r) is one of the expert's.
constexpr bool tile_has_row(int32_t row0, int32_t row_end, int32_t r) { return r < row_end - row0; }

// The tile's row r, or past the expert's end its last row.
constexpr int32_t tile_row(int32_t row0, int32_t row_end, int32_t r) {
  return row0 + (tile_has_row(row0, row_end, r) ? r : row_end - row0 - 1);
}

}  // namespace moe
