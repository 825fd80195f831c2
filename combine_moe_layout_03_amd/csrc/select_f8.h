// Which kernel a call of the 8-bit float products takes.  Host arithmetic only,
// without HIP, so that a CPU test can compile it.
#pragma once

#include <stdint.h>

namespace moe {
namespace select {

enum class GemmF8Kind { kStream32, kTile64, kTile128, kTile256 };

// Workgroups to expect: every other expert ends inside a tile.
constexpr int64_t gemm_f8_workgroups(int32_t rows, int32_t groups, int32_t n, int tile_m, int tile_n) {
  return (rows / tile_m + (int64_t(groups) + 1) / 2) * ((int64_t(n) + tile_n - 1) / tile_n);
}
constexpr GemmF8Kind gemm_f8_kind(int32_t rows, int32_t groups, int32_t n) {
  const int64_t mean = (int64_t(rows) + groups - 1) / groups;
  if (mean <= 16) return GemmF8Kind::kStream32;
  if (mean > 128 && gemm_f8_workgroups(rows, groups, n, 256, 256) >= 128) return GemmF8Kind::kTile256;
  if (mean > 48 && gemm_f8_workgroups(rows, groups, n, 128, 128) >= 128) return GemmF8Kind::kTile128;
  return gemm_f8_workgroups(rows, groups, n, 64, 128) >= 128 ? GemmF8Kind::kTile64 : GemmF8Kind::kStream32;
}
constexpr GemmF8Kind gemm_f8_gated_kind(int32_t rows, int32_t groups, int32_t n) {
  const int64_t mean = (int64_t(rows) + groups - 1) / groups;
  if (mean <= 16) return GemmF8Kind::kStream32;
  if (mean > 96 && gemm_f8_workgroups(rows, groups, n, 128, 128) >= 128) return GemmF8Kind::kTile128;
  return gemm_f8_workgroups(rows, groups, n, 64, 128) >= 128 ? GemmF8Kind::kTile64 : GemmF8Kind::kStream32;
}

}  // namespace select
}  // namespace moe
