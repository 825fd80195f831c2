// Which kernel a call of the 8-bit float products takes.  Host arithmetic only,
// without HIP, so that a CPU test can compile it.
#pragma once

#include <stdint.h>

namespace moe {
namespace select {

// The rows an expert has on average (when all have some, and the counts add up
// to the call's rows: the host does not know less) decide how many rows a tile
// takes, measured at 16 experts whose counts fall as rank^-1/2 (us, bf16
// results; tile32, tile64, tile256):
//   k 2048, n 7168, 16 rows: 40, 41, 63       k 7168, n 2048, 24 rows: 42, 42, 77
//   200: 45, 46, 67                           200: 43, 43, 78
//   400: 54, 49, 68                           768: 57, 68, 85
//   1500: 91, 74, 76                          3000: 153, 114, 101
//   3000: 143, 108, 101
//   6000: 244, 179, 140
// The widened products (fp32 results) have a tile of 256 x 128 in the place of
// tile256, and fewer workgroups than about 256 of 256 x 256 are slower with it
// (tile64, tile256: 32768 rows, k 2048, n 7168: 1158, 1012; 16384, k and n 2048, 4
// experts, 528 workgroups: 168, 159; 8000, k 4096, n 1024, 8 experts, 140: 92,
// 110; 8-bit products 60, 47).
//
// Few workgroups of 16 columns are the fastest (split16; three a CU fit on the
// chip at once, 768): 2 rows, 8 experts, k 5904, n 213: 7.8, the best of the others
// 23; 30, 5, 5488, 1546: 13.8, 22; 1000, 1, 7168, 128: 14.3, 23.  By their number
// (split16 and the best of the others at k 2048; at k 7168):
//   640 (64 rows, 1 expert, n 2048): 8.0, 9.7; 17.3, 22.9
//   880 (64, 1, 2816): 8.1, 9.5; 18.1, 22.8
//   1020 (64, 1, 3264): 10.3, 9.8; 23.4, 22.9
//   1024 (8, 8, 2048): 10.8, 9.5; 30.4, 32.1
//   1280 (64, 1, 4096): 11.5, 9.8; 27.2, 23.0
//   1408 (300, 4, 1024): 13.0, 9.8; 31.7, 29.8
// The widened tiles are slower, and for them the limit is low: 1024: 11.1, 14.6;
// 30.4, 41.8; 1280: 11.4, 15.0; 27.3, 40.7; 1408: 12.8, 15.1; 32.1, 41.1.
enum class GemmF8Kind { kSplit16, kTile32, kTile64, kTile256 };

// Workgroups to expect: every other expert ends inside a tile.
constexpr int64_t gemm_f8_workgroups(int32_t rows, int32_t groups, int32_t n, int tile_m, int tile_n) {
  return (rows / tile_m + (int64_t(groups) + 1) / 2) * ((int64_t(n) + tile_n - 1) / tile_n);
}
// The workgroups of 16 columns (a quarter of k to each of their four waves).
constexpr int64_t gemm_f8_split_workgroups(int32_t rows, int32_t groups, int32_t n) {
  return (rows / 16 + int64_t(rows < groups ? rows : groups)) * ((int64_t(n) + 15) / 16);
}
constexpr int64_t gemm_f8_mean(int32_t rows, int32_t groups) { return (int64_t(rows) + groups - 1) / groups; }
constexpr GemmF8Kind gemm_f8_kind(int32_t rows, int32_t groups, int32_t n, bool wide) {
  const int64_t mean = gemm_f8_mean(rows, groups);
  if (gemm_f8_split_workgroups(rows, groups, n) <= 1024) return GemmF8Kind::kSplit16;
  if (mean <= 16) return GemmF8Kind::kTile32;
  if (mean > 128 && gemm_f8_workgroups(rows, groups, n, 256, 256) >= (wide ? 256 : 128)) return GemmF8Kind::kTile256;
  return GemmF8Kind::kTile64;
}

// The gated product of few rows passes its activations through a workspace, as
// floats, to a kernel that quantises them: its workgroups need not hold whole
// blocks of 128 columns then, and fill the chip (8 rows, 8 experts, k 7168, n
// 2048: 47 us, and 71 with 128 columns a workgroup).  With more rows for each
// expert, and workgroups enough, a workgroup of 128 x 128 quantises its own (3000
// rows, 16 experts: 230 us, and 264 through the workspace; 1500: 193, 165; 4000,
// 4 experts, k and n 512: 19, 15).
//
// The workspace ends at 4096 rows, 16 KB for each column.  Past it many experts of
// few rows pay for tiles that they do not fill, the others do not (us, tiles of
// 128 x 128, and through a workspace of all rows; n 2048): 4112 rows, 128 experts,
// k 2048: 334, 255; 8192, 256, 2048: 668, 511; 8192, 128, 7168: 1096, 955; but
// 8192, 64, 7168: 694, 778; 6000, 40, 7168: 468, 534; 16384, 128, 7168: 1397, 1563.
constexpr int32_t kF8ActRows = 4096;
constexpr bool gemm_f8_act(int32_t rows, int32_t groups, int32_t n) {
  return rows <= kF8ActRows &&
         (gemm_f8_mean(rows, groups) <= 128 || gemm_f8_workgroups(rows, groups, n, 128, 128) < 192);
}
// As above (k 7168, n 2048, 16 experts, us; tile32, tile64: 24 rows 84, 92; 200:
// 87, 93; 400: 121, 95; 768: 125, 124; 1500: 199, 165; but short rows of weights
// suit the smaller tile, 777 rows, 7 experts, n 1008: k 1040 17.1, 20.7; 7168 53.6,
// 66.1).  With two reads of weights for each column split16 (two a CU, 512) up to
// fewer workgroups (split16 and the best tile at k 2048; at k 7168): 576 (30 rows,
// 5 experts, n 1536) 13.0, 18.3; 29.1, 45.5; 768 (8, 8, 1536) 18.3, 19.3; 43.9,
// 45.9; 800 (64, 1, 2560) 15.3, 18.4; 34.5, 45.5; 896 (8, 8, 1792) 20.0, 19.2; 47.1,
// 45.9; 1024 (8, 8, 2048) 21.0, 19.6; 48.7, 46.2.
constexpr GemmF8Kind gemm_f8_act_kind(int32_t rows, int32_t groups, int32_t n) {
  if (gemm_f8_split_workgroups(rows, groups, n) <= 768) return GemmF8Kind::kSplit16;
  return gemm_f8_mean(rows, groups) <= 16 ? GemmF8Kind::kTile32 : GemmF8Kind::kTile64;
}

}  // namespace select
}  // namespace moe
