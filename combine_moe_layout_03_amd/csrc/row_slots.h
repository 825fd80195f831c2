// Experts' rows from device-side counts: expert g owns the rows [S_g, S_g +
// c_g), c_g = max(count_g, 0) and S_g the sum of the counts before g, cut at
// `rows`.  A launch that works on tiles of TM rows numbers the experts' tiles
// ("row slots") in order; a wave finds the rows of a slot here.
#pragma once

#include "device_util.h"

namespace moe {

struct RowSlot {
  int32_t group, row0, row_end;
};

// Row slots enough for any counts: expert g needs at most c_g / TM + 1 tiles,
// and at most `rows` experts have a row.
inline int64_t row_slots(int32_t rows, int32_t groups, int tile_rows) {
  return (static_cast<int64_t>(rows) + tile_rows - 1) / tile_rows + (rows < groups ? rows : groups);
}

// One wave, all of it active; the result is the same in every lane.  Counts
// are clipped to `rows` and summed with saturation: a sum that saturates is
// past `rows` (below 2^31) whatever is added or taken away after it.
template <int TM>
__device__ __forceinline__ bool find_row_slot(const int32_t* counts, int groups, int rows, int64_t slot, int lane,
                                              RowSlot* out) {
  const auto add_sat = [](int x, int y) {
    return static_cast<int>(__builtin_elementwise_add_sat(static_cast<uint32_t>(x), static_cast<uint32_t>(y)));
  };
  const uint32_t limit = static_cast<uint32_t>(rows);
  uint32_t row_base = 0;
  int64_t tile_base = 0;
  for (int g0 = 0; g0 < groups; g0 += kWave) {
    const int g = g0 + lane;
    const uint32_t c = g < groups ? static_cast<uint32_t>(min(max(counts[g], 0), rows)) : 0u;
    const uint32_t incl = static_cast<uint32_t>(wave_scan_dpp(static_cast<int>(c), add_sat));
    const uint32_t s = min(static_cast<uint32_t>(add_sat(static_cast<int>(row_base), static_cast<int>(incl - c))), limit);
    const uint32_t e = min(static_cast<uint32_t>(add_sat(static_cast<int>(row_base), static_cast<int>(incl))), limit);
    const int tiles = static_cast<int>((e - s + TM - 1) / TM);
    const int tincl = wave_inclusive_scan(tiles);
    const int64_t t0 = tile_base + tincl - tiles;
    const uint64_t hit = __ballot(slot >= t0 && slot < t0 + tiles);
    if (hit != 0) {
      const int l = __builtin_ctzll(hit);
      out->group = g0 + l;
      out->row0 = __builtin_amdgcn_readlane(static_cast<int>(s + static_cast<uint32_t>(slot - t0) * TM), l);
      out->row_end = __builtin_amdgcn_readlane(static_cast<int>(e), l);
      return true;
    }
    row_base = min(static_cast<uint32_t>(add_sat(static_cast<int>(row_base), __builtin_amdgcn_readlane(static_cast<int>(incl), kWave - 1))), limit);
    tile_base += __builtin_amdgcn_readlane(tincl, kWave - 1);
    if (row_base >= limit) break;
  }
  return false;
}

}  // namespace moe
