// Arguments and launchers of the block-scaled 8-bit float expert products.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"

namespace moe {

// What becomes of the sums: rounded to a type, or gated and quantised.
// (kAct: gated, as binary32, for the workspace of a gated call)
enum class Form { kBf16 = 0, kFp16 = 1, kF32 = 2, kGated = 3, kAct = 4 };

// Bytes between rows at most: a tile's rows lie within 32-bit offsets.
constexpr int64_t kF8MaxRowBytes = int64_t(1) << 23;

struct GemmF8Args {
  const uint8_t* a;            // row m at a + m * a_stride, k e4m3 codes
  int64_t a_stride;            // bytes between rows (a multiple of 16)
  int32_t rows;
  int32_t k;                   // a multiple of 16
  const int32_t* group_count;  // [groups]
  int32_t groups;
  const uint8_t* w;            // [groups][n][k], with SwiGLU [groups][2n][k]
  int32_t n;                   // columns of the result
  const float* weight_scale;   // [groups][blocks of n][blocks of k], with SwiGLU [groups][2 blocks of n][blocks of k]
  const uint8_t* token_scale;  // blocks of k floats of row m from byte m * ts_stride on
  int64_t ts_stride;
  void* out;                   // [rows][n]; with SwiGLU e4m3 rows of out_row_bytes
  int64_t out_row_bytes;
  int32_t out_scale_off;
  void* workspace;             // of a gated call of few rows: the activations, float [rows][n]
  bool nt;                     // set by the launcher: the tiles' results are stored non-temporally
};
// Whether one launch holds the call's threads.
bool grouped_gemm_f8_fits(int32_t rows, int32_t groups, int32_t n, Form form);
hipError_t launch_grouped_gemm_f8(GemmF8Args a, Form form, hipStream_t stream);

}  // namespace moe
