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

// Sums of counts saturate: a sum that does is past `rows` (below 2^31)
// whatever is added or taken away after it.
__device__ __forceinline__ uint32_t add_sat(uint32_t x, uint32_t y) { return __builtin_elementwise_add_sat(x, y); }

// The rows and slots of 64 experts from g0, one for each lane.
template <int TM>
struct SlotLanes {
  uint32_t s, e;      // the expert's rows
  int32_t tiles, t0;  // its slots, and the first of them past the experts before g0
  uint32_t rows_end;  // rows of the experts up to these (the same in every lane)
  int32_t count;      // slots of these 64 experts (the same in every lane)
};
template <int TM>
__device__ __forceinline__ SlotLanes<TM> slot_lanes(const int32_t* counts, int groups, int rows, int g0,
                                                    uint32_t row_base, int lane) {
  const auto sat = [](int x, int y) {
    return static_cast<int>(add_sat(static_cast<uint32_t>(x), static_cast<uint32_t>(y)));
  };
  const uint32_t limit = static_cast<uint32_t>(rows);
  const int g = g0 + lane;
  const uint32_t c = g < groups ? static_cast<uint32_t>(min(max(counts[g], 0), rows)) : 0u;
  const uint32_t incl = static_cast<uint32_t>(wave_scan_dpp(static_cast<int>(c), sat));
  SlotLanes<TM> l;
  l.s = min(add_sat(row_base, incl - c), limit);
  l.e = min(add_sat(row_base, incl), limit);
  l.tiles = static_cast<int32_t>((l.e - l.s + TM - 1) / TM);
  const int tincl = wave_inclusive_scan(l.tiles);
  l.t0 = tincl - l.tiles;
  l.rows_end = min(add_sat(row_base, static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(incl), kWave - 1))), limit);
  l.count = __builtin_amdgcn_readlane(tincl, kWave - 1);
  return l;
}

// Slot `slot` (counted from these experts' first) if it is one of theirs.
template <int TM>
__device__ __forceinline__ bool take_slot(const SlotLanes<TM>& l, int g0, int64_t slot, RowSlot* out) {
  const uint64_t hit = __ballot(slot >= l.t0 && slot < l.t0 + l.tiles);
  if (hit == 0) return false;
  const int q = __builtin_ctzll(hit);
  out->group = g0 + q;
  out->row0 = __builtin_amdgcn_readlane(static_cast<int>(l.s + static_cast<uint32_t>(slot - l.t0) * TM), q);
  out->row_end = __builtin_amdgcn_readlane(static_cast<int>(l.e), q);
  return true;
}

// The rows of slot `slot` (the same in every lane; the whole wave active).
// False if there are fewer slots.
template <int TM>
__device__ __forceinline__ bool find_row_slot(const int32_t* counts, int groups, int rows, int64_t slot, int lane,
                                              RowSlot* out) {
  uint32_t row_base = 0;
  for (int g0 = 0; g0 < groups; g0 += kWave) {
    const SlotLanes<TM> l = slot_lanes<TM>(counts, groups, rows, g0, row_base, lane);
    if (slot < l.count) return take_slot(l, g0, slot, out);
    slot -= l.count;
    row_base = l.rows_end;
    if (row_base >= static_cast<uint32_t>(rows)) break;
  }
  return false;
}

// The same for a slot that depends on how many slots the counts give: pick
// (slots) is the slot, or -1 for none.
template <int TM, typename Pick>
__device__ __forceinline__ bool place_row_slot(const int32_t* counts, int groups, int rows, int lane, Pick pick,
                                               RowSlot* out) {
  const SlotLanes<TM> l = slot_lanes<TM>(counts, groups, rows, 0, 0, lane);
  int64_t total = l.count;
  uint32_t row_base = l.rows_end;
  for (int g0 = kWave; g0 < groups && row_base < static_cast<uint32_t>(rows); g0 += kWave) {
    const SlotLanes<TM> m = slot_lanes<TM>(counts, groups, rows, g0, row_base, lane);
    total += m.count;
    row_base = m.rows_end;
  }
  const int64_t slot = pick(total);
  if (slot < 0) return false;
  if (slot < l.count) return take_slot(l, 0, slot, out);
  return find_row_slot<TM>(counts, groups, rows, slot, lane, out);
}

}  // namespace moe
