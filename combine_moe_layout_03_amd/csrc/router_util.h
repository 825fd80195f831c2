// Device helpers of the router and its gradient: wave reductions, logits of
// three types, and the selection keys.
#pragma once

#include <float.h>

#include "device_util.h"
#include "launch.h"

namespace moe {

template <Out kType>
__device__ __forceinline__ float load_float(const void* base, int64_t i) {
  if constexpr (kType == Out::kF32) {
    return static_cast<const float*>(base)[i];
  } else {
    return half_to_f32<kType == Out::kFp16>(static_cast<const uint16_t*>(base)[i]);
  }
}

template <Out kType>
__device__ __forceinline__ void store_float(void* base, int64_t i, float v) {
  if constexpr (kType == Out::kF32) {
    static_cast<float*>(base)[i] = v;
  } else {
    static_cast<uint16_t*>(base)[i] =
        static_cast<uint16_t>(kType == Out::kFp16 ? f32_to_f16(v) : f32_to_bf16(v));
  }
}

// A product rounded to binary32 before it is converted to binary16: left to
// itself the compiler folds the two into v_fma_mixlo_f16, which rounds the
// exact product once (another result now and then).
__device__ __forceinline__ float round_f32(float v) {
  asm("" : "+v"(v));
  return v;
}

// A logit as the router reads it: -inf for an expert that is not eligible
// (-inf, NaN), +inf as the largest finite value, -0 as +0.
__device__ __forceinline__ float router_logit(float v) {
  const float x = v > -__builtin_inff() ? v : -__builtin_inff();  // NaN fails the comparison
  return (x < FLT_MAX ? x : FLT_MAX) + 0.0f;
}

__device__ __forceinline__ float wave_sum_f32(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}
__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v = __builtin_fmaxf(v, __shfl_xor(v, d, kWave));
  return v;
}

// 1 / (1 + e^-x) without an overflow on either side.
__device__ __forceinline__ float sigmoid_f32(float x) {
  const float e = expf(-__builtin_fabsf(x));
  return (x > 0.0f ? 1.0f : e) / (1.0f + e);
}

// The chosen scores over a common factor that makes the largest of them at
// least 1/2, so their ratios hold where the scores underflow: e^(x - m) for
// the softmax (m the largest chosen logit), and for the sigmoid e^(x - c) / (1
// + e^x) with c = min(m, 0), which for x > 0 (then c = 0) is 1 / (1 + e^-x).
template <bool kSigmoid>
__device__ __forceinline__ float relative_score(float x, float m) {
  if constexpr (!kSigmoid) return expf(x - m);
  return x > 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x - __builtin_fminf(m, 0.0f)) / (1.0f + expf(x));
}

}  // namespace moe
