// The gradient of the combine: for the entries (t, j) of token t, with g its
// output gradient and y the entry's receive row,
//   row gradient = round(w_tj * g),   weight gradient = sum_i y[i] * g[i].
//
// One workgroup per token.  A thread owns chunks of 8 elements and takes the
// token's entries eight at a time: per chunk it reads g once and each entry's
// y, adds to the entry's sum and stores the entry's row gradient, so a row
// may be replaced in place.  A sum is one thread's chunks in order, then the
// lanes of a wave, then the waves: a fixed order.
#include "device_util.h"
#include "launch.h"
#include "router_util.h"

#pragma clang fp contract(off)

namespace moe {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kGroup = 8;  // entries taken together

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <bool kFp16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (kFp16) return f32_to_f16(round_f32(a)) | (f32_to_f16(round_f32(b)) << 16);
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

template <bool kFp16>
__device__ __forceinline__ void widen(const u32x4& w, float (&f)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    f[2 * q] = half_to_f32<kFp16>(w[q] & 0xffffu);
    f[2 * q + 1] = half_to_f32<kFp16>(w[q] >> 16);
  }
}

template <Out kGrad>
__device__ __forceinline__ void load_grad(const void* base, int64_t elem, float (&f)[8]) {
  if constexpr (kGrad == Out::kF32) {
    const f32x4* p = reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + elem);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int q = 0; q < 4; ++q) f[q] = a[q], f[4 + q] = b[q];
  } else {
    widen<kGrad == Out::kFp16>(*reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(base) + elem), f);
  }
}

template <bool kFp16, Out kGrad>
__global__ __launch_bounds__(kThreads) void combine_backward_kernel(RouteArgs a, const void* grad_out,
                                                                    const uint8_t* recv, const float* topk_w,
                                                                    uint8_t* grad_recv, float* grad_w) {
  __shared__ float part[kWaves][kGroup];
  const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
  const int t = blockIdx.x;
  const int chunks = a.hidden >> 3;
  for (int j0 = 0; j0 < a.k; j0 += kGroup) {
    int64_t off[kGroup];
    bool valid[kGroup];
    float w[kGroup], sum[kGroup];
    resolve_rows<kGroup>(a, t, j0, lane, off, valid);
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      w[j] = topk_w[static_cast<int64_t>(t) * a.k + min(j0 + j, a.k - 1)];
      sum[j] = 0.0f;
    }
    for (int c = tid; c < chunks; c += kThreads) {
      float g[8];
      load_grad<kGrad>(grad_out, static_cast<int64_t>(t) * a.hidden + c * 8, g);
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        if (!valid[j]) continue;
        float y[8];
        widen<kFp16>(*reinterpret_cast<const u32x4*>(recv + off[j] + c * 16), y);
#pragma unroll
        for (int q = 0; q < 8; ++q) sum[j] = __builtin_fmaf(y[q], g[q], sum[j]);
        u32x4 d;
#pragma unroll
        for (int q = 0; q < 4; ++q) d[q] = pack2<kFp16>(w[j] * g[2 * q], w[j] * g[2 * q + 1]);
        *reinterpret_cast<u32x4*>(grad_recv + off[j] + c * 16) = d;
      }
    }
    __syncthreads();  // the previous entries' sums have been read
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) sum[j] += __shfl_xor(sum[j], d, kWave);
      if (lane == 0) part[wave][j] = sum[j];
    }
    __syncthreads();
    if (tid < kGroup && j0 + tid < a.k) {
      float s = part[0][tid];
#pragma unroll
      for (int q = 1; q < kWaves; ++q) s += part[q][tid];
      grad_w[static_cast<int64_t>(t) * a.k + j0 + tid] = s;
    }
  }
}

template <bool kFp16>
hipError_t launch_grad(const RouteArgs& r, const void* grad_out, Out grad_type, const uint8_t* recv,
                       const float* topk_w, uint8_t* grad_recv, float* grad_w, hipStream_t stream) {
  const dim3 grid(static_cast<unsigned>(r.bs)), block(kThreads);
#define MOE_CASE(G)                                                                                             \
  case G:                                                                                                       \
    hipLaunchKernelGGL((combine_backward_kernel<kFp16, G>), grid, block, 0, stream, r, grad_out, recv, topk_w,  \
                       grad_recv, grad_w);                                                                      \
    return hipGetLastError();
  switch (grad_type) {
    MOE_CASE(Out::kBf16)
    MOE_CASE(Out::kFp16)
    MOE_CASE(Out::kF32)
  }
#undef MOE_CASE
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_combine_backward(const RouteArgs& r, const void* grad_out, Out grad_type, const void* recv_x,
                                   Half recv_type, const float* topk_w, void* grad_recv, float* grad_weights,
                                   hipStream_t stream) {
  const uint8_t* recv = static_cast<const uint8_t*>(recv_x);
  uint8_t* grad = static_cast<uint8_t*>(grad_recv);
  return recv_type == Half::kFp16
             ? launch_grad<true>(r, grad_out, grad_type, recv, topk_w, grad, grad_weights, stream)
             : launch_grad<false>(r, grad_out, grad_type, recv, topk_w, grad, grad_weights, stream);
}

}  // namespace moe
