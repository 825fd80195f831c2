// Shapes of the norm's kernels.  Host arithmetic only, without HIP, so that a
// CPU test can compile it.
#pragma once

#include <stdint.h>

namespace moe {
namespace select {

// A row's chunks of 8 elements are dealt to the lanes of `waves` waves, at most
// `chunks` to a lane (1, 2 or 4).  Rows of one wave stand four in a workgroup.
struct NormShape {
  int chunks, waves;
};
constexpr int kNormRowsPerGroup = 4;  // of one wave each
constexpr int norm_waves(int32_t hidden, int chunks) { return (hidden / 8 + 64 * chunks - 1) / (64 * chunks); }
constexpr NormShape norm_shape(int32_t, int32_t hidden) {
  const int chunks = hidden <= 512 ? 1 : hidden <= 8192 ? 2 : 4;
  return NormShape{chunks, norm_waves(hidden, chunks)};
}
constexpr NormShape norm_backward_shape(int32_t, int32_t hidden) { return norm_shape(0, hidden); }

// Rows of one launch: fewer than 2^32 threads at up to 16 waves a row.
constexpr int32_t kNormLaunchRows = int32_t(1) << 21;

// Parts of the batch whose weight gradients are summed on their own first.
constexpr int32_t kNormBackwardParts = 512;
constexpr int32_t norm_backward_parts(int32_t bs) { return bs < kNormBackwardParts ? bs : kNormBackwardParts; }

}  // namespace select
}  // namespace moe
