// Arguments and launchers of the root-mean-square norm and its gradient.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "select_norm.h"

namespace moe {

struct NormArgs {
  const void* x;         // [bs][hidden]
  const void* residual;  // [bs][hidden] or null
  const float* weight;   // [hidden]
  float eps;
  int32_t bs, hidden;
  void* sum;             // [bs][hidden] of x's type, or null
  void* out;             // [bs][hidden] of out_type, or null
  Out out_type;
  uint8_t* rows;         // e4m3 rows, or null
  int64_t row_bytes;
  int32_t scale_off;
  float* rstd;           // [bs] or null
};
hipError_t launch_rms_norm(const NormArgs& a, Out type, hipStream_t stream);

struct NormBackwardArgs {
  const void* grad_out;  // [bs][hidden]
  const void* grad_sum;  // [bs][hidden] of sum's type, or null
  const void* sum;       // [bs][hidden]
  const float* weight;   // [hidden]
  const float* rstd;     // [bs]
  const uint8_t* token_mask;  // [bs] or null
  int32_t bs, hidden;
  void* grad_x;          // [bs][hidden] of sum's type
  float* grad_weight;    // [hidden] or null
  float* partial;        // [norm_backward_parts(bs, hidden)][hidden] where grad_weight is given
};
hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, Out type, Out grad_type, hipStream_t stream);

}  // namespace moe
