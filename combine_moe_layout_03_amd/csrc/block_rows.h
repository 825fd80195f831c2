// 8-bit float rows: e4m3 codes and a float scale for each 128 of them
// (include/moe_ep.h, MOE_E4M3_BLOCKSCALE).  A block of values y becomes
//   d = max(max |y|, 2^-100), scale = d / 448, code = e4m3(y * (448 / d))
// with binary32 divisions and product, and one rounding to 8 bits (half to
// even).  448 is e4m3's largest value; |y| (448 / d) is at most 448 (1 + 2^-22),
// far from 464, where rounding would leave the range.  The floor keeps 448 / d
// finite where a block is zero or nearly so (its codes are then 0 or small).
#pragma once

#include "device_util.h"

namespace moe {

constexpr int kF8Block = 128;         // columns (and elements of k) that share a scale
constexpr float kF8Largest = 448.0f;  // of e4m3
constexpr float kF8Tiny = 0x1p-100f;

__host__ __device__ constexpr int32_t f8_blocks(int32_t width) { return (width + kF8Block - 1) / kF8Block; }

// Scale of a block whose largest magnitude is amax, and the factor of its codes.
__device__ __forceinline__ void f8_scale(float amax, float& scale, float& factor) {
  const float d = __builtin_fmaxf(amax, kF8Tiny);
  scale = d / kF8Largest;
  factor = kF8Largest / d;
}

// Codes of four values (already multiplied), the first in the lowest byte.
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  return static_cast<uint32_t>(v);
}

typedef int32_t i32x2 __attribute__((ext_vector_type(2)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float mfma_f32x4 __attribute__((ext_vector_type(4)));

// 16 x 16 products over 128 codes.  A lane holds 32 codes of an operand's row,
// two pieces of 16; the same pieces of both operands meet, so which 16 they are
// does not matter.  The first operand's rows run along a lane's four results.
//
// Widened to bf16, which holds every e4m3 value, the products are exact and
// summed in binary32.
struct WideCodes {
  bf16x8 v[4];
};
__device__ __forceinline__ bf16x8 widen(i32x2 codes) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x8 w;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const bf16x2 two = q & 1 ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[q / 2], 1.0f, true)
                             : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes[q / 2], 1.0f, false);
    w[2 * q] = two[0], w[2 * q + 1] = two[1];
  }
  return w;
}
__device__ __forceinline__ WideCodes widen(i32x4 a, i32x4 b) {
  return WideCodes{{widen(i32x2{a[0], a[1]}), widen(i32x2{a[2], a[3]}), widen(i32x2{b[0], b[1]}),
                    widen(i32x2{b[2], b[3]})}};
}
// The 8-bit instruction, as it stands.
__device__ __forceinline__ mfma_f32x4 block_sum(const i32x8& a, const i32x8& b) {
  constexpr int kE4m3 = 0;
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, mfma_f32x4{0.0f, 0.0f, 0.0f, 0.0f}, kE4m3, kE4m3, 0, 0,
                                                          0, 0);
}
__device__ __forceinline__ i32x8 join(i32x4 a, i32x4 b) {
  return i32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ mfma_f32x4 block_sum(const WideCodes& a, const WideCodes& b) {
  mfma_f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < 4; ++q) p = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[q], b.v[q], p, 0, 0, 0);
  return p;
}

}  // namespace moe
