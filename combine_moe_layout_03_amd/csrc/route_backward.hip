// The router's gradient: the gradient of the weights carried back to the
// logits (the choice is constant).  With a_j = s_j / Z the chosen shares,
//   renormalised weights: dx_j = scale a_j (g_j - sum_i g_i a_i) at the chosen
//     experts, times 1 - s_j for the sigmoid, and 0 elsewhere (for the softmax
//     the shares are the softmax of the chosen logits alone);
//   else, sigmoid: dx_j = scale g_j s_j (1 - s_j) at the chosen experts;
//   else, softmax: dx_e = p_e (scale g_e - sum_i scale g_i p_i), every expert.
//
// A token is the work of 16 lanes or of a wave, as in route.hip: lane j < k
// works on entry j and puts its value at the expert's place in a row of LDS,
// which the lanes cleared or, for the last formula, filled.  Bound by the bytes:
// 16384 tokens x 256 experts, fp32, sigmoid: 5.2 us for 17 MB of gradients and
// the lines of the chosen logits (12 MB); the last formula reads all of them (8.7
// us, where its bytes take 5.6).
#include "device_util.h"
#include "layer.h"
#include "router_util.h"

namespace moe {
namespace {

constexpr int kWaves = 4;

template <bool kSigmoid, int kL, int kVpl>
__global__ __launch_bounds__(kWaves* kWave) void route_backward_kernel(RouterArgs a, Out type) {
  constexpr int kTokens = kWave / kL;
  __shared__ __attribute__((aligned(16))) float rows[kWaves * kTokens][kL * kVpl];
  const int lane = threadIdx.x % kL, sub = threadIdx.x / kL;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (kTokens * kWaves) + sub;
  const bool active = token < a.bs;
  const int64_t t = active ? token : a.bs - 1;  // lanes past the batch work on its last token and store nothing
  const int64_t row = t * a.stride;
  using Row = TokenRow<kL, kVpl>;
  float* place = rows[sub];
  const bool dense = !kSigmoid && !a.renorm;  // every expert's logit has a gradient
  float p[kVpl];
#pragma unroll
  for (int i = 0; i < kVpl; ++i) p[i] = 0.0f;
  if (!dense) Row::put(place, lane, p);

  int id = -1;
  float xm = -__builtin_inff(), g = 0.0f;
  if (lane < a.k) {
    const int64_t o = t * a.k + lane;
    id = a.topk_idx[o];
    if (static_cast<unsigned>(id) < static_cast<unsigned>(a.num_experts))
      xm = router_logit(load_logit(a.logits, type, row + id));
    if (xm > -__builtin_inff()) g = a.grad_weights[o] * a.scale;
    else id = -1;
  }

  float ds = 0.0f;
  if (dense) {
    float x[kVpl];
    Row::load(a.logits, type, row, a.num_experts, lane, place);
    wave_lds_sync();
    Row::get(place, lane, x);
    float top = x[0], sum = 0.0f;
#pragma unroll
    for (int i = 1; i < kVpl; ++i) top = __builtin_fmaxf(top, x[i]);
    top = token_max<kL>(top);
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      p[i] = x[i] > -__builtin_inff() ? expf(x[i] - top) : 0.0f;
      sum += p[i];
    }
    sum = token_sum<kL>(sum);
    if (sum == 0.0f) sum = 1.0f;  // no eligible expert: p is 0
    ds = id >= 0 ? g * (expf(xm - top) / sum) : 0.0f;
    const float dot = token_sum<kL>(ds);
#pragma unroll
    for (int i = 0; i < kVpl; ++i) p[i] = p[i] > 0.0f ? -(p[i] / sum) * dot : 0.0f;  // 0 also where dot is not finite
    wave_lds_sync();
    Row::put(place, lane, p);
  } else if (a.renorm) {
    const float m = token_max<kL>(xm);
    const float r = id >= 0 ? relative_score<kSigmoid>(xm, m) : 0.0f;
    const float z = token_sum<kL>(r);
    const float share = id >= 0 ? r / z : 0.0f;
    ds = share * (g - token_sum<kL>(g * share));
    if (kSigmoid) ds *= id >= 0 ? sigmoid_f32(-xm) : 0.0f;
  } else {
    if (id >= 0) ds = g * (sigmoid_f32(xm) * sigmoid_f32(-xm));
  }
  wave_lds_sync();
  if (id >= 0) place[Row::at(id)] += ds;
  wave_lds_sync();
  if (active) Row::store(a.grad_logits, type, token * a.grad_stride, a.num_experts, lane, place);
}

template <bool kSigmoid, int kL, int kVpl>
hipError_t launch_shape(const RouterArgs& a, Out type, hipStream_t stream) {
  constexpr int kTokens = kWave / kL * kWaves;
  const dim3 grid(static_cast<unsigned>((a.bs + kTokens - 1) / kTokens)), block(kWaves * kWave);
  hipLaunchKernelGGL((route_backward_kernel<kSigmoid, kL, kVpl>), grid, block, 0, stream, a, type);
  return hipGetLastError();
}

template <bool kSigmoid>
hipError_t launch_score(const RouterArgs& a, Out type, hipStream_t stream) {
  return with_router_shape(select::router_shape(a.bs, a.num_experts, a.k), [&](auto lanes, auto vpl) {
    return launch_shape<kSigmoid, decltype(lanes)::value, decltype(vpl)::value>(a, type, stream);
  });
}

}  // namespace

hipError_t launch_route_backward(const RouterArgs& a, Out logits_type, bool sigmoid, hipStream_t stream) {
  for (int64_t first = 0; first < a.bs; first += select::router_launch_tokens()) {
    const RouterArgs part = router_part(a, logits_type, static_cast<int32_t>(first));
    const hipError_t e =
        sigmoid ? launch_score<true>(part, logits_type, stream) : launch_score<false>(part, logits_type, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
