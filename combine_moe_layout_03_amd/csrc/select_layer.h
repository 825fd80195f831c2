// Which variant a call of the router, of the gradients and of the second expert
// matmul takes.  Host arithmetic only, without HIP, so that a CPU test can
// compile it.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moe {
namespace select {

// ---- second expert matmul: kernel and tile ----------------------------------
// The kernel and tile of a call.  The rows an expert has on average (when all
// have some, and the counts add up to the call's rows: the host does not know
// less) decide how many rows a tile takes, measured at 16 experts whose
// counts fall as rank^-1/2 (us; stream16, stream32, tile64, tile128, tile256):
//   k 2048, n 7168, 24 rows: 44, 44, 46       k 7168, n 2048, 16 rows: 41, 42, 48
//   64: 46, 47, 47                            128: 55, 56, 51
//   200: 51, 49, 46                           200: 55, 58, 51
//   512: -, 63, 48, 51, 64                    768: -, 76, 60, 53, 63
//   1500: -, 119, 75, 68, 66                  3000: -, 209, 110, 94, 95 (k 2048)
// Fewer than about half as many workgroups as there are CUs leave the chip
// idle, and then the next smaller tile is the faster one (777 rows, k 1040, n
// 1001, 7 experts, 128 workgroups of tile64 by the estimate below: 22 us with
// tile256, 16, 11, 8.6 with stream32; 1000 rows, k 4096, n 1024, 8 experts, 152
// of tile64: 36 with tile256, 21, 19 with tile64, 30 with stream32; 8000 such
// rows, 140 of tile256: 44 with tile256, 53 with tile128).  kFewTile64 lies
// between the first two of these, which differ in k as well.
//
// Where all workgroups of 16 columns fit on the chip at once (four a CU), those
// are the fastest (split16, and the best of the others; us): 2 rows, 8 experts,
// k 5904, n 213: 6.9, 10.6; 30, 5, 5488, 1546: 12.5, 12.9; 128, 4, 7168, 512:
// 11.7, 18.8; 1000, 1, 7168, 128: 13.4, 20.0; 24, 12, 7168, 1024 (832 of them):
// 20.4, 21.8; but 128, 2, 4096, 2048 (1280): 15.0, 13.0.
enum class GemmDeqKind { kStream16, kStream32, kTile64, kTile128, kTile256, kSplit16 };

// Workgroups to expect: every other expert ends inside a tile.
constexpr int64_t gemm_deq_workgroups(int32_t rows, int32_t groups, int32_t n, int tile_m, int tile_n) {
  return (rows / tile_m + (int64_t(groups) + 1) / 2) * ((int64_t(n) + tile_n - 1) / tile_n);
}
constexpr GemmDeqKind gemm_deq_kind(int32_t rows, int32_t groups, int32_t n) {
  constexpr int64_t kFewWorkgroups = 128, kFewTile64 = 144, kSplitWorkgroups = 1024;
  const int64_t slots16 = rows / 16 + (rows < groups ? rows : groups);
  if (slots16 * ((int64_t(n) + 15) / 16) <= kSplitWorkgroups) return GemmDeqKind::kSplit16;
  const int64_t mean = (int64_t(rows) + groups - 1) / groups;
  if (mean <= 4) return GemmDeqKind::kStream16;
  if (mean > 128 && gemm_deq_workgroups(rows, groups, n, 256, 256) >= kFewWorkgroups) return GemmDeqKind::kTile256;
  if (mean > 48 && gemm_deq_workgroups(rows, groups, n, 128, 128) >= kFewWorkgroups) return GemmDeqKind::kTile128;
  return gemm_deq_workgroups(rows, groups, n, 64, 128) >= kFewTile64 ? GemmDeqKind::kTile64 : GemmDeqKind::kStream32;
}

// The streams' chunks of k: 256 bytes end nearer to a short k, 512 have half the
// barriers; stream16 takes the 512 as two parts of 256, each the work of two of
// its waves (us, 256, 512 and two parts; stream16, 48 rows: k 512 8.5, 9.4, -, k
// 768 13.4, 16.4, 16.7, k 1024 30.9, 30.9, 30.1, 64 rows: k 2048 48.1, 46.2, 44.0,
// 24 rows: k 7168 -, 81.0, 76.9; stream32: k 1040 7.8, 8.5, k 1536 7.3, 7.3, k
// 2048 9.9, 8.4, k 4112 16.2, 15.9).
constexpr bool gemm_deq_short_chunks(GemmDeqKind kind, int32_t k) {
  return k < (kind == GemmDeqKind::kStream16 ? 1024 : 1536);
}

// Results of the tiles: non-temporally where weights, rows and results are more
// than the caches keep, so that they do not push the weights out; else the next
// kernel finds them there (bf16, and with a kernel that reads them after it, us,
// non-temporally and not: 1001 x 512 weights of 8 experts and 3001 rows, 12 MB,
// 8.9 + 7.0 and 9.0 + 5.2; 1024 x 4096, 8 and 1000, 40 MB, 19.0 + 2.4, 18.9 +
// 2.2; 7168 x 2048, 16 and 1000, 251 MB, 54.8 + 6.1, 58.8 + 7.4; 32768 rows,
// 772 MB, 465 + 137, 471 + 138).
constexpr int64_t kGemmDeqNtBytes = int64_t(64) << 20;
constexpr bool gemm_deq_nt(int64_t rows, int64_t groups, int64_t k, int64_t n, int out_size) {
  return groups * n * k + rows * (k + n * out_size) > kGemmDeqNtBytes;
}

// ---- combine's gradient: how the row gradients are stored --------------------
// Non-temporally where the rows are more than the caches keep (h 7168, 8
// entries, bf16, non-temporal and not: 512 tokens, 59 MB of rows: 25.3 and
// 24.1 us; 768: 37.8, 35.0; 1024: 48.8, 52.3; 4096: 198, 210).
constexpr int64_t kCombineBackwardNtBytes = int64_t(96) << 20;
constexpr bool combine_backward_nt(int64_t row_bytes) { return row_bytes > kCombineBackwardNtBytes; }
// Short rows: 16 lanes an entry, four a wave (16 lanes and a wave, 4096 tokens, 8
// entries, bf16, us: h 64 4.6 and 9.5, h 256 8.7, 14.2, h 512 14.4, 17.5, h 1024
// 26.2, 26.2; 61 tokens, 5, h 1000: 3.9, 2.5).  Rows past kCombineBackwardNtBytes
// take a wave all the same (8 entries, h 256, 16384 and 32768 tokens: 26, 90).
constexpr bool combine_backward_short(int32_t hidden) { return hidden <= 512; }

// ---- router and its gradient: (lanes of a token, experts of a lane) -----------
// 16 lanes a token, four tokens a wave, where a row of 16 holds the experts
// and the entries and the batch is large (the choice among 256 experts by
// either: 1024 tokens 5.0 and, a wave each, 4.8 us; 2048: 5.0, 5.7; 4096: 5.2,
// 8.1; 16384: 13.2, 23.8); else a wave.
struct RouterShape {
  int lanes, vpl;
};
constexpr RouterShape kRouterShapes[] = {{16, 1}, {16, 2}, {16, 4}, {16, 8}, {16, 16}, {64, 1},
                                         {64, 2}, {64, 4}, {64, 8}, {64, 16}, {64, 32}};
constexpr int kRouterRowTokens = 2048;
constexpr RouterShape router_shape(int bs, int experts, int topk) {
  const int lanes = topk <= 16 && experts <= 256 && bs >= kRouterRowTokens ? 16 : 64;
  for (const RouterShape s : kRouterShapes)
    if (s.lanes == lanes && s.lanes * s.vpl >= experts) return s;
  return RouterShape{0, 0};
}

// ---- tokens of one launch ------------------------------------------------------
// A launch has fewer than 2^32 threads, and the router and the gradients give
// up to a wave to a token or an entry; a larger batch is launched in parts.
constexpr int32_t kLaunchWaves = int32_t(1) << 25;
constexpr int32_t router_launch_tokens() { return kLaunchWaves; }
constexpr int32_t combine_backward_launch_tokens(int32_t topk) { return kLaunchWaves / topk; }

}  // namespace select
}  // namespace moe
