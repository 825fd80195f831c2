// Helpers of the router, of the gradients and of the second expert matmul:
// vector types and 16-bit pairs, logits of three types, reductions over a
// token's lanes, a token's row through LDS, and the launch by the router's shape.
#pragma once

#include <float.h>

#include <type_traits>
#include <utility>

#include "device_util.h"
#include "launch.h"
#include "select_layer.h"

namespace moe {

// f(lanes, vpl) with the shape as compile-time constants; one instance of f for
// each of select::kRouterShapes.
template <typename F, size_t... I>
hipError_t with_router_shape(select::RouterShape s, F f, std::index_sequence<I...>) {
  hipError_t e = hipErrorInvalidValue;
  const auto is = [&](select::RouterShape t) { return s.lanes == t.lanes && s.vpl == t.vpl; };
  ((is(select::kRouterShapes[I]) ? void(e = f(std::integral_constant<int, select::kRouterShapes[I].lanes>{},
                                              std::integral_constant<int, select::kRouterShapes[I].vpl>{}))
                                 : void()),
   ...);
  return e;
}
template <typename F>
hipError_t with_router_shape(select::RouterShape s, F f) {
  constexpr size_t kCount = sizeof(select::kRouterShapes) / sizeof(select::kRouterShapes[0]);
  return with_router_shape(s, f, std::make_index_sequence<kCount>{});
}

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

// ---- a token's lanes ------------------------------------------------------------
// A token is the work of kL lanes, 16 (a DPP row; four tokens a wave) or 64;
// lane l holds the kVpl experts from l * kVpl.  All of a wave's lanes stay
// active: the reductions read their neighbours.

// Exchanges that pair the lanes of a row so that four steps reach all 16:
// lane ^ 1, lane ^ 2, then the mirrors of 8 and of 16 lanes (after the steps
// before them every lane of the other half holds the same value).
constexpr int kDppXor1 = 0xb1, kDppXor2 = 0x4e, kDppMirror8 = 0x141, kDppMirror16 = 0x140;

template <int kCtrl>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kCtrl, 0xf, 0xf, true));
}
template <int kCtrl>
__device__ __forceinline__ double dpp(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(b & 0xffffffffu), kCtrl, 0xf, 0xf, true));
  const uint32_t hi =
      static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), kCtrl, 0xf, 0xf, true));
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}
__device__ __forceinline__ float lane_value(float v, int q) { return lane_float(v, q); }
__device__ __forceinline__ double lane_value(double v, int q) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b & 0xffffffffu), q));
  const uint32_t hi = static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(b >> 32), q));
  return __builtin_bit_cast(double, (static_cast<uint64_t>(hi) << 32) | lo);
}

// op over the token's lanes, in every one of them (the same order for each).
template <int kL, typename T, typename Op>
__device__ __forceinline__ T token_reduce(T v, Op op) {
  static_assert(kL == 16 || kL == 64, "a row or the wave");
  v = op(v, dpp<kDppXor1>(v));
  v = op(v, dpp<kDppXor2>(v));
  v = op(v, dpp<kDppMirror8>(v));
  v = op(v, dpp<kDppMirror16>(v));
  if constexpr (kL == 64)
    v = op(op(lane_value(v, 0), lane_value(v, 16)), op(lane_value(v, 32), lane_value(v, 48)));
  return v;
}
template <int kL, typename T>
__device__ __forceinline__ T token_sum(T v) {
  return token_reduce<kL>(v, [](T a, T b) { return a + b; });
}
template <int kL>
__device__ __forceinline__ float token_max(float v) {
  return token_reduce<kL>(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
template <int kL>
__device__ __forceinline__ double token_max(double v) {
  return token_reduce<kL>(v, [](double a, double b) { return __builtin_fmax(a, b); });
}

// Orders this wave's LDS writes before its later LDS reads of other lanes' data.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// Accesses at any element's address (a row of an odd length starts anywhere).
typedef f32x4 f32x4_u __attribute__((aligned(4)));
typedef u32x2 u32x2_u __attribute__((aligned(2)));
typedef u32x4 u32x4_u __attribute__((aligned(2)));

// Two values rounded to 16 bits, the first in the lower half.
template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (kFp16) return f32_to_f16(round_f32(a)) | (f32_to_f16(round_f32(b)) << 16);
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ float load_logit(const void* base, Out type, int64_t i) {
  if (type == Out::kF32) return load_float<Out::kF32>(base, i);
  return type == Out::kFp16 ? load_float<Out::kFp16>(base, i) : load_float<Out::kBf16>(base, i);
}

// The logits from element i on, kN of them (of which `have` exist; the others
// read as -inf), as the router reads them.
template <int kN>
__device__ __forceinline__ void load_logits(const void* base, Out type, int64_t i, int have, float (&x)[kN]) {
  if (kN % 4 == 0 && have >= kN) {
    if (type == Out::kF32) {
#pragma unroll
      for (int q = 0; q < kN / 4; ++q) {
        const f32x4 v = *reinterpret_cast<const f32x4_u*>(static_cast<const float*>(base) + i + 4 * q);
#pragma unroll
        for (int r = 0; r < 4; ++r) x[4 * q + r] = v[r];
      }
    } else {
      uint32_t w[kN / 2 > 0 ? kN / 2 : 1];
      const uint16_t* p = static_cast<const uint16_t*>(base) + i;
      if constexpr (kN % 8 == 0) {
#pragma unroll
        for (int q = 0; q < kN / 8; ++q) {
          const u32x4 v = *reinterpret_cast<const u32x4_u*>(p + 8 * q);
#pragma unroll
          for (int r = 0; r < 4; ++r) w[4 * q + r] = v[r];
        }
      } else if constexpr (kN % 4 == 0) {
        const u32x2 v = *reinterpret_cast<const u32x2_u*>(p);
        w[0] = v[0], w[1] = v[1];
      }
#pragma unroll
      for (int q = 0; q < kN; ++q) {
        const uint32_t b = (q & 1) ? w[q / 2] >> 16 : w[q / 2] & 0xffffu;
        x[q] = type == Out::kFp16 ? f16_to_f32(b) : bf16_to_f32(b);
      }
    }
#pragma unroll
    for (int q = 0; q < kN; ++q) x[q] = router_logit(x[q]);
  } else {
#pragma unroll
    for (int q = 0; q < kN; ++q)
      x[q] = q < have ? router_logit(load_logit(base, type, i + q)) : -__builtin_inff();
  }
}

// ---- a token's row through LDS ----------------------------------------------------
// Global memory is read and written in 16-byte pieces that lie side by side in
// a wave's lanes; the work is on kVpl neighbours a lane.  LDS is where the two
// meet: a row of kL kVpl floats.  (Rows of 256 fp32 gradients stored 64 bytes a
// lane: 10.1 us for 16384 of them; in pieces side by side 6.6, non-temporally
// 5.7.  The choice, which only reads, is as fast with its loads a lane's own.)
template <int kL, int kVpl>
struct TokenRow {
  static constexpr int kSize = kL * kVpl;
  // Place of element e: where a lane has 16 neighbours, the four pieces of lanes
  // 4 apart change places, so that 16 lanes reading one piece each meet all banks.
  static __device__ __forceinline__ int at(int e) { return kVpl == 16 ? e ^ ((e >> 4) & 12) : e; }

  // Logits of the row from element `row` on, as router_logit() gives them, and
  // -inf past the experts.
  static __device__ __forceinline__ void load(const void* base, Out type, int64_t row, int experts, int lane,
                                              float* lds) {
    if (type == Out::kF32) {
      constexpr int kRounds = (kVpl + 3) / 4;
      f32x4 v[kRounds];
#pragma unroll
      for (int q = 0; q < kRounds; ++q) {  // every load before the first use
        const int e = (q * kL + lane) * 4;
        if (e + 4 <= experts) {
          v[q] = *reinterpret_cast<const f32x4_u*>(static_cast<const float*>(base) + row + e);
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            v[q][r] = e + r < experts ? load_float<Out::kF32>(base, row + e + r) : -__builtin_inff();
        }
      }
#pragma unroll
      for (int q = 0; q < kRounds; ++q) {
        const int e = (q * kL + lane) * 4;
        if (e < kSize) put4(lds, e, v[q]);
      }
    } else {
      constexpr int kRounds = (kVpl + 7) / 8;
      u32x4 w[kRounds];
#pragma unroll
      for (int q = 0; q < kRounds; ++q) {
        const int e = (q * kL + lane) * 8;
        const uint16_t* p = static_cast<const uint16_t*>(base) + row + e;
        if (e + 8 <= experts) {
          w[q] = *reinterpret_cast<const u32x4_u*>(p);
        } else {
          const uint32_t none = type == Out::kFp16 ? 0xfc00u : 0xff80u;  // -inf
#pragma unroll
          for (int r = 0; r < 4; ++r)
            w[q][r] = (e + 2 * r < experts ? p[2 * r] : none) | ((e + 2 * r + 1 < experts ? p[2 * r + 1] : none) << 16);
        }
      }
#pragma unroll
      for (int q = 0; q < kRounds; ++q) {
        const int e = (q * kL + lane) * 8;
        float f[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const uint32_t b = (r & 1) ? w[q][r / 2] >> 16 : w[q][r / 2] & 0xffffu;
          f[r] = type == Out::kFp16 ? f16_to_f32(b) : bf16_to_f32(b);
        }
        if (e < kSize) put4(lds, e, f32x4{f[0], f[1], f[2], f[3]});
        if (e + 4 < kSize) put4(lds, e + 4, f32x4{f[4], f[5], f[6], f[7]});
      }
    }
  }
  static __device__ __forceinline__ void put4(float* lds, int e, f32x4 v) {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = router_logit(v[r]);
    if (kSize % 4 == 0) {
      *reinterpret_cast<f32x4*>(lds + at(e)) = v;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (e + r < kSize) lds[e + r] = v[r];
    }
  }

  // This lane's neighbours.
  static __device__ __forceinline__ void get(const float* lds, int lane, float (&x)[kVpl]) {
    if constexpr (kVpl % 4 == 0) {
#pragma unroll
      for (int q = 0; q < kVpl / 4; ++q) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(lds + at(lane * kVpl + 4 * q));
#pragma unroll
        for (int r = 0; r < 4; ++r) x[4 * q + r] = v[r];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVpl; ++i) x[i] = lds[lane * kVpl + i];
    }
  }
  static __device__ __forceinline__ void put(float* lds, int lane, const float (&x)[kVpl]) {
    if constexpr (kVpl % 4 == 0) {
#pragma unroll
      for (int q = 0; q < kVpl / 4; ++q)
        *reinterpret_cast<f32x4*>(lds + at(lane * kVpl + 4 * q)) =
            f32x4{x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]};
    } else {
#pragma unroll
      for (int i = 0; i < kVpl; ++i) lds[lane * kVpl + i] = x[i];
    }
  }

  // The row's elements, rounded to `type`, to element `row` on.
  static __device__ __forceinline__ void store(void* base, Out type, int64_t row, int experts, int lane,
                                               const float* lds) {
    if (type == Out::kF32) {
#pragma unroll
      for (int q = 0; q < (kVpl + 3) / 4; ++q) {
        const int e = (q * kL + lane) * 4;
        if (e + 4 <= experts) {
          f32x4 v;
          if constexpr (kSize % 4 == 0) v = *reinterpret_cast<const f32x4*>(lds + at(e));
          __builtin_nontemporal_store(v, reinterpret_cast<f32x4_u*>(static_cast<float*>(base) + row + e));
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (e + r < experts) store_float<Out::kF32>(base, row + e + r, lds[at(e + r)]);
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < (kVpl + 7) / 8; ++q) {
        const int e = (q * kL + lane) * 8;
        uint16_t* p = static_cast<uint16_t*>(base) + row + e;
        uint32_t h[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) {
          const float f = e + r < experts ? lds[at(e + r)] : 0.0f;
          h[r] = type == Out::kFp16 ? f32_to_f16(round_f32(f)) : f32_to_bf16(f);
        }
        if (e + 8 <= experts) {
          __builtin_nontemporal_store(
              u32x4{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)},
              reinterpret_cast<u32x4_u*>(p));
        } else {
#pragma unroll
          for (int r = 0; r < 8; ++r)
            if (e + r < experts) p[r] = static_cast<uint16_t>(h[r]);
        }
      }
    }
  }
};

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
