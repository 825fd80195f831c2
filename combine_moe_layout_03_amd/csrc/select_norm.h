// Shapes of the norm's kernels.  Host arithmetic only, without HIP, so that a
// CPU test can compile it.
#pragma once

#include <stdint.h>

namespace moe {
namespace select {

// A row's chunks of 8 elements are dealt to the lanes of `waves` waves, at most
// `chunks` to a lane: 1 in one wave, 2 in one wave or up to 8, 4 in up to 8.
// Rows of one wave stand four in a workgroup.
// (4096 tokens, h 7168, bf16, one, two or four chunks a lane: 51.3, 51.0, 51.4
// us; the gradient, 68.6, 68.3, 68.2: two, for fewer waves at the barrier.)
struct NormShape {
  int chunks, waves;
};
constexpr int kNormRowsPerGroup = 4;  // of one wave each
constexpr NormShape norm_shape(int32_t hidden) {
  const int chunks = hidden <= 512 ? 1 : hidden <= 8192 ? 2 : 4;
  return NormShape{chunks, (hidden / 8 + 64 * chunks - 1) / (64 * chunks)};
}

// Rows of one launch: fewer than 2^32 threads at up to 8 waves a row.
constexpr int32_t kNormLaunchRows = int32_t(1) << 21;

// Loads: non-temporal where the call reads more than the caches keep (h 7168,
// bf16, us, non-temporal and not: 512 tokens 8.5, 6.8; 2048, 59 MB read: 26.2,
// 20.7; 4096, 117 MB: 47.2, 49.5; 8192: 88.3, 93.9; the gradient, 2048, 88 MB:
// 27.4, 25.7; 4096: 45.9, 46.3; 8192: 81.9, 83.9).
constexpr int64_t kNormNtBytes = int64_t(96) << 20;
constexpr bool norm_nt(int64_t read_bytes) { return read_bytes > kNormNtBytes; }

// The gradient: rows of a workgroup, as many as eight waves hold, and parts of
// the batch whose weight gradients are summed on their own first (4096 tokens,
// h 7168, bf16, 128, 256, 512 and 1024 parts: 56, 44, 50, 90 us).
constexpr int32_t kNormBackwardParts = 256;
constexpr int kNormJoinedHidden = 4096;  // columns of a row of at most four waves
constexpr int32_t norm_backward_rows(int waves) { return waves > 4 ? 1 : 8 / waves; }
constexpr int32_t norm_backward_parts(int32_t bs, int32_t hidden) {
  const int64_t rows = norm_backward_rows(norm_shape(hidden).waves);
  const int64_t sets = (bs + rows - 1) / rows;
  return static_cast<int32_t>(sets < kNormBackwardParts ? sets : kNormBackwardParts);
}

}  // namespace select
}  // namespace moe
