// The router's gradient: the gradient of the weights carried back to the
// logits (the choice is constant).  With a_j = s_j / Z the chosen shares,
//   renormalised weights: dx_j = scale a_j (g_j - sum_i g_i a_i) at the chosen
//     experts, times 1 - s_j for the sigmoid, and 0 elsewhere (for the softmax
//     the shares are the softmax of the chosen logits alone);
//   else, sigmoid: dx_j = scale g_j s_j (1 - s_j) at the chosen experts;
//   else, softmax: dx_e = p_e (scale g_e - sum_i scale g_i p_i), every expert.
// One wave per token: lane j < k works on entry j, then lane l writes the
// experts l + 64 i, i < kVpl.
#include "device_util.h"
#include "launch.h"
#include "router_util.h"

namespace moe {
namespace {

constexpr int kBackwardWaves = 4;

template <Out kType, bool kSigmoid, int kVpl>
__global__ __launch_bounds__(kBackwardWaves* kWave) void route_backward_kernel(RouterArgs a) {
  const int lane = threadIdx.x % kWave, wave = uniform(static_cast<int>(threadIdx.x / kWave));
  const int t = static_cast<int>(blockIdx.x) * kBackwardWaves + wave;
  if (t >= a.bs) return;
  const int64_t row = t * a.stride;

  int id = -1;
  float xm = -__builtin_inff(), g = 0.0f;
  if (lane < a.k) {
    const int64_t o = static_cast<int64_t>(t) * a.k + lane;
    id = a.topk_idx[o];
    if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_experts))
      xm = router_logit(load_float<kType>(a.logits, row + id));
    if (xm > -__builtin_inff()) g = a.grad_weights[o] * a.scale;
    else id = -1;
  }

  float ds = 0.0f, dot = 0.0f, top = 0.0f, sum = 1.0f;
  float p[kVpl];
#pragma unroll
  for (int i = 0; i < kVpl; ++i) p[i] = 0.0f;
  if (a.renorm) {
    const float m = wave_max_f32(xm);
    const float r = id >= 0 ? relative_score<kSigmoid>(xm, m) : 0.0f;
    const float z = wave_sum_f32(r);
    const float share = id >= 0 ? r / z : 0.0f;
    ds = share * (g - wave_sum_f32(g * share));
    if (kSigmoid) ds *= id >= 0 ? sigmoid_f32(-xm) : 0.0f;
  } else if (kSigmoid) {
    if (id >= 0) ds = g * (sigmoid_f32(xm) * sigmoid_f32(-xm));
  } else {
    float x[kVpl];
    top = -__builtin_inff();
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      const int e = lane + i * kWave;
      x[i] = e < a.num_experts ? router_logit(load_float<kType>(a.logits, row + e)) : -__builtin_inff();
      top = __builtin_fmaxf(top, x[i]);
    }
    top = wave_max_f32(top);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      p[i] = x[i] > -__builtin_inff() ? expf(x[i] - top) : 0.0f;
      sum += p[i];
    }
    sum = wave_sum_f32(sum);
    if (sum == 0.0f) sum = 1.0f;  // no eligible expert: p is 0
    ds = id >= 0 ? g * (expf(xm - top) / sum) : 0.0f;
    dot = wave_sum_f32(ds);
#pragma unroll
    for (int i = 0; i < kVpl; ++i) p[i] = -(p[i] / sum) * dot;
  }
#pragma unroll
  for (int i = 0; i < kVpl; ++i) {
    const int e = lane + i * kWave;
    float d = p[i];
    for (int j = 0; j < a.k; ++j)
      if (__builtin_amdgcn_readlane(id, j) == e) d += lane_float(ds, j);
    if (e < a.num_experts) store_float<kType>(a.grad_logits, t * a.grad_stride + e, d);
  }
}

template <Out kType, bool kSigmoid>
hipError_t launch_vpl(const RouterArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>((a.bs + kBackwardWaves - 1) / kBackwardWaves)), block(kBackwardWaves * kWave);
#define MOE_ROUTE_CASE(V)                                                                          \
  case V:                                                                                          \
    hipLaunchKernelGGL((route_backward_kernel<kType, kSigmoid, V>), grid, block, 0, stream, a);    \
    return hipGetLastError();
  switch (select::router_vpl(a.num_experts)) {
    MOE_ROUTE_CASE(1)
    MOE_ROUTE_CASE(2)
    MOE_ROUTE_CASE(4)
    MOE_ROUTE_CASE(8)
    MOE_ROUTE_CASE(16)
    MOE_ROUTE_CASE(32)
  }
#undef MOE_ROUTE_CASE
  return hipErrorInvalidValue;
}

template <Out kType>
hipError_t launch_score(const RouterArgs& a, bool sigmoid, hipStream_t stream) {
  return sigmoid ? launch_vpl<kType, true>(a, stream) : launch_vpl<kType, false>(a, stream);
}

}  // namespace

hipError_t launch_route_backward(const RouterArgs& a, Out logits_type, bool sigmoid, hipStream_t stream) {
  switch (logits_type) {
    case Out::kBf16: return launch_score<Out::kBf16>(a, sigmoid, stream);
    case Out::kFp16: return launch_score<Out::kFp16>(a, sigmoid, stream);
    case Out::kF32: return launch_score<Out::kF32>(a, sigmoid, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
