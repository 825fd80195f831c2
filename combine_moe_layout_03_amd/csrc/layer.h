// Arguments and launchers of the router, of the gradients and of the second
// expert matmul.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.h"
#include "select_layer.h"

namespace moe {

// ---- router and the gradients of the routed path ----------------------------------
struct RouterArgs {
  const void* logits;         // row t at element t * stride
  int64_t stride;
  int32_t bs, num_experts, k;
  const float* bias;          // [E] or null
  int32_t groups, keep, group_top, group_size;
  uint64_t group_magic;       // div_magic(group_size)
  int32_t renorm;
  float scale;
  const uint8_t* token_mask;  // [bs] or null
  int32_t* topk_idx;          // [bs, k] (read by the gradient)
  float* topk_weights;        // [bs, k]
  // the gradient
  const float* grad_weights;  // [bs, k]
  void* grad_logits;          // row t at element t * grad_stride
  int64_t grad_stride;
};
// The call's tokens from `first` on, as many as one launch takes.
inline RouterArgs router_part(RouterArgs a, Out logits_type, int32_t first) {
  const int64_t es = logits_type == Out::kF32 ? 4 : 2, at = first;
  a.bs = a.bs - first < select::router_launch_tokens() ? a.bs - first : select::router_launch_tokens();
  a.logits = static_cast<const uint8_t*>(a.logits) + at * a.stride * es;
  a.topk_idx += at * a.k;
  if (a.topk_weights != nullptr) a.topk_weights += at * a.k;
  if (a.token_mask != nullptr) a.token_mask += at;
  if (a.grad_weights != nullptr) a.grad_weights += at * a.k;
  if (a.grad_logits != nullptr) a.grad_logits = static_cast<uint8_t*>(a.grad_logits) + at * a.grad_stride * es;
  return a;
}
hipError_t launch_route(const RouterArgs& a, Out logits_type, bool sigmoid, hipStream_t stream);
hipError_t launch_route_backward(const RouterArgs& a, Out logits_type, bool sigmoid, hipStream_t stream);
hipError_t launch_combine_backward(const RouteArgs& r, const void* grad_out, Out grad_type, const void* recv_x,
                                   Half recv_type, const float* topk_w, void* grad_recv, float* grad_weights,
                                   hipStream_t stream);

// ---- second expert matmul: int8 products, scaled to 16- or 32-bit floats ----------
struct GemmDeqArgs {
  const int8_t* a;             // row m at a + m * a_stride, k int8 codes
  int64_t a_stride;            // bytes between rows (a multiple of 16)
  int32_t rows;
  int32_t k;                   // a multiple of 16
  const int32_t* group_count;  // [groups]
  int32_t groups;
  const int8_t* w;             // [groups][n][k]
  int32_t n;
  const float* weight_scale;   // [groups][n]
  const uint8_t* token_scale;  // float of row m at byte m * ts_stride
  int64_t ts_stride;
  void* out;                   // [rows][n]
  bool nt;                     // set by the launcher: the tiles' results are stored non-temporally
};
// Whether one launch holds the call's threads.
bool grouped_gemm_deq_fits(int32_t rows, int32_t groups, int32_t n);
hipError_t launch_grouped_gemm_deq(GemmDeqArgs a, Out out_type, hipStream_t stream);

}  // namespace moe
