// Which kernel a call of the 8-bit float products takes.  Host arithmetic only,
// without HIP, so that a CPU test can compile it.
#pragma once

#include <stdint.h>

namespace moe {
namespace select {

enum class GemmF8Kind { kSplit16, kTile32, kTile64, kTile256 };

// Workgroups to expect: every other expert ends inside a tile.
constexpr int64_t gemm_f8_workgroups(int32_t rows, int32_t groups, int32_t n, int tile_m, int tile_n) {
  return (rows / tile_m + (int64_t(groups) + 1) / 2) * ((int64_t(n) + tile_n - 1) / tile_n);
}
// The workgroups of 16 columns (a quarter of k to each of their four waves).
constexpr int64_t gemm_f8_split_workgroups(int32_t rows, int32_t groups, int32_t n) {
  return (rows / 16 + int64_t(rows < groups ? rows : groups)) * ((int64_t(n) + 15) / 16);
}
constexpr GemmF8Kind gemm_f8_kind(int32_t rows, int32_t groups, int32_t n) {
  const int64_t mean = (int64_t(rows) + groups - 1) / groups;
  if (gemm_f8_split_workgroups(rows, groups, n) <= 1024) return GemmF8Kind::kSplit16;
  if (mean <= 16) return GemmF8Kind::kTile32;
  if (mean > 128 && gemm_f8_workgroups(rows, groups, n, 256, 256) >= 128) return GemmF8Kind::kTile256;
  return GemmF8Kind::kTile64;
}

constexpr int32_t kF8ActRows = 4096;
constexpr bool gemm_f8_act(int32_t rows, int32_t groups, int32_t n) {
  const int64_t mean = (int64_t(rows) + groups - 1) / groups;
  return rows <= kF8ActRows && (mean <= 128 || gemm_f8_workgroups(rows, groups, n, 128, 128) < 192);
}
constexpr GemmF8Kind gemm_f8_act_kind(int32_t rows, int32_t groups, int32_t n) {
  const int64_t mean = (int64_t(rows) + groups - 1) / groups;
  if (gemm_f8_split_workgroups(rows, groups, n) <= 768) return GemmF8Kind::kSplit16;
  return mean <= 16 ? GemmF8Kind::kTile32 : GemmF8Kind::kTile64;
}

}  // namespace select
}  // namespace moe
