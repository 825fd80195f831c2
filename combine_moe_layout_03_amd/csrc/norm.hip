// Root-mean-square norm with the residual's addition, in front of the router
// and the dispatch, and its gradient.  For a row x of a token
//   s = round(x + residual), rstd = 1 / sqrt(mean(s^2) + eps), y = (s rstd) w
//   out = round(y), and 8-bit rows of y (block_rows.h)
// Sums are binary32: a lane's chunks in order, then the lanes, then the waves.
//
// A row's chunks of 8 elements lie in the registers of its lanes from the load
// to the stores, so every element is read and written once.  16 neighbouring
// lanes hold the 128 columns of an 8-bit block.
#include "block_rows.h"
#include "device_util.h"
#include "norm.h"
#include "router_util.h"

#pragma clang fp contract(off)

namespace moe {
namespace {

constexpr int kMaxWaves = 16;
// Of a workgroup (select::norm_shape keeps to it; more of them would leave a lane too few registers).
constexpr int max_waves(int chunks) { return chunks == 1 ? kMaxWaves : 8; }

// Eight elements as they lie in memory.
template <Out kType>
struct Chunk {
  u32x4 w[kType == Out::kF32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t elem) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(base) +
                                                    elem * (kType == Out::kF32 ? 4 : 2));
    w[0] = p[0];
    if constexpr (kType == Out::kF32) w[1] = p[1];
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if constexpr (kType == Out::kF32) f[q] = __uint_as_float(w[q / 4][q % 4]);
      else f[q] = half_to_f32<kType == Out::kFp16>((q & 1) ? w[0][q / 2] >> 16 : w[0][q / 2] & 0xffffu);
    }
  }
  // f rounded to the type, here and in f.
  __device__ __forceinline__ void round(float (&f)[8]) {
    if constexpr (kType == Out::kF32) {
#pragma unroll
      for (int q = 0; q < 8; ++q) w[q / 4][q % 4] = __float_as_uint(f[q]);
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) w[0][q] = pack2<kType == Out::kFp16>(f[2 * q], f[2 * q + 1]);
      get(f);
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t elem) const {
    u32x4* p = reinterpret_cast<u32x4*>(static_cast<uint8_t*>(base) + elem * (kType == Out::kF32 ? 4 : 2));
    p[0] = w[0];
    if constexpr (kType == Out::kF32) p[1] = w[1];
  }
};

template <Out kType>
__device__ __forceinline__ void store_rounded(void* base, int64_t elem, float (&f)[8]) {
  Chunk<kType> c;
  c.round(f);
  c.store(base, elem);
}

__device__ __forceinline__ void load_weight(const float* weight, int col, float (&w)[8]) {
  const f32x4_u* p = reinterpret_cast<const f32x4_u*>(weight + col);
  const f32x4 a = p[0], b = p[1];
#pragma unroll
  for (int q = 0; q < 4; ++q) w[q] = a[q], w[4 + q] = b[q];
}

// The sum of v over the row's waves, in every lane.
template <bool kOneWave>
__device__ __forceinline__ float row_sum(float v, int waves, float* lds) {
  v = token_sum<kWave>(v);
  if constexpr (kOneWave) return v;
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  float s = 0.0f;
  for (int q = 0; q < waves; ++q) s += lds[q];
  return s;
}

template <Out kType, int kChunks, bool kOneWave>
__global__ __launch_bounds__(kOneWave ? kWave* select::kNormRowsPerGroup : kWave* max_waves(kChunks)) void rms_norm_kernel(
    NormArgs a) {
  __shared__ float lds[kMaxWaves];
  const int waves = kOneWave ? 1 : blockDim.x / kWave;
  const int t = kOneWave ? blockIdx.x * select::kNormRowsPerGroup + uniform(threadIdx.x / kWave) : blockIdx.x;
  if (t >= a.bs) return;  // a wave, or the whole workgroup
  const int lane = kOneWave ? threadIdx.x % kWave : threadIdx.x, lanes = waves * kWave;
  const int chunks = a.hidden / 8;
  const int64_t row = static_cast<int64_t>(t) * a.hidden;
  Chunk<kType> x[kChunks], r[kChunks];
  float w[kChunks][8];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {  // (past the row's end its last chunk, which counts for nothing)
    const int c = min(lane + i * lanes, chunks - 1);
    x[i].load(a.x, row + c * 8);
    if (a.residual != nullptr) r[i].load(a.residual, row + c * 8);
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) load_weight(a.weight, min(lane + i * lanes, chunks - 1) * 8, w[i]);
  float y[kChunks][8], squares = 0.0f;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const bool mine = lane + i * lanes < chunks;
    x[i].get(y[i]);
    if (a.residual != nullptr) {
      float f[8];
      r[i].get(f);
#pragma unroll
      for (int q = 0; q < 8; ++q) y[i][q] += f[q];
      x[i].round(y[i]);
    }
    if (mine) {
      if (a.sum != nullptr) x[i].store(a.sum, row + (lane + i * lanes) * 8);
#pragma unroll
      for (int q = 0; q < 8; ++q) squares = __builtin_fmaf(y[i][q], y[i][q], squares);
    }
  }
  squares = row_sum<kOneWave>(squares, waves, lds);
  const float rstd = 1.0f / __builtin_sqrtf(squares / static_cast<float>(a.hidden) + a.eps);
  if (a.rstd != nullptr && lane == 0) a.rstd[t] = rstd;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int c = lane + i * lanes;
    const bool mine = c < chunks;
    float amax = 0.0f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      y[i][q] = y[i][q] * rstd * w[i][q];
      amax = __builtin_fmaxf(amax, __builtin_fabsf(y[i][q]));
    }
    if (a.rows != nullptr) {
      float scale, factor;
      f8_scale(token_max<16>(mine ? amax : 0.0f), scale, factor);
      if (mine) {
        uint8_t* dst = a.rows + t * a.row_bytes;
        float f[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = y[i][q] * factor;
        *reinterpret_cast<u32x2*>(dst + c * 8) =
            u32x2{f8_pack4(f[0], f[1], f[2], f[3]), f8_pack4(f[4], f[5], f[6], f[7])};
        if (c % 16 == 0) *reinterpret_cast<float*>(dst + a.scale_off + c / 16 * 4) = scale;
      }
    }
    if (a.out != nullptr && mine) {
      if (a.out_type == Out::kF32) store_rounded<Out::kF32>(a.out, row + c * 8, y[i]);
      else if (a.out_type == Out::kFp16) store_rounded<Out::kFp16>(a.out, row + c * 8, y[i]);
      else store_rounded<Out::kBf16>(a.out, row + c * 8, y[i]);
    }
  }
}

// The gradient.  With xh = s rstd and gw = g w
//   dx = rstd (gw - xh mean(gw xh)) + dsum,  dw = sum over the tokens of g xh
// A workgroup takes every parts-th row; a lane has the same columns of each, so
// its part of dw stays in registers, is written once and summed by the second
// kernel, in a fixed order.
template <Out kType, Out kGrad, int kChunks, bool kOneWave>
__global__ __launch_bounds__(kOneWave ? kWave : kWave* max_waves(kChunks)) void rms_norm_backward_kernel(NormBackwardArgs a) {
  __shared__ float lds[2][kMaxWaves];
  const int waves = kOneWave ? 1 : blockDim.x / kWave;
  const int lane = threadIdx.x, lanes = waves * kWave;
  const int chunks = a.hidden / 8;
  float w[kChunks][8], dw[kChunks][8];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    load_weight(a.weight, min(lane + i * lanes, chunks - 1) * 8, w[i]);
#pragma unroll
    for (int q = 0; q < 8; ++q) dw[i][q] = 0.0f;
  }
  const float mean = 1.0f / static_cast<float>(a.hidden);
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.bs; t += gridDim.x) {
    const int64_t row = t * a.hidden;
    if (a.token_mask != nullptr && a.token_mask[t] == 0) {  // the same in every lane
      float zero[8] = {};
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        if (lane + i * lanes < chunks) store_rounded<kType>(a.grad_x, row + (lane + i * lanes) * 8, zero);
      continue;
    }
    Chunk<kGrad> gc[kChunks];
    Chunk<kType> sc[kChunks], skip[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int c = min(lane + i * lanes, chunks - 1);
      gc[i].load(a.grad_out, row + c * 8);
      sc[i].load(a.sum, row + c * 8);
      if (a.grad_sum != nullptr) skip[i].load(a.grad_sum, row + c * 8);
    }
    const float rstd = a.rstd[t];
    float g[kChunks][8], xh[kChunks][8], dot = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      gc[i].get(g[i]);
      sc[i].get(xh[i]);
      const bool mine = lane + i * lanes < chunks;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        xh[i][q] *= rstd;
        dw[i][q] = __builtin_fmaf(g[i][q], xh[i][q], dw[i][q]);
        g[i][q] *= w[i][q];
        if (mine) dot = __builtin_fmaf(g[i][q], xh[i][q], dot);
      }
    }
    dot = row_sum<kOneWave>(dot, waves, lds[turn]) * mean;
    turn ^= 1;  // the other sums may still be read
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      float f[8], s[8] = {};
      if (a.grad_sum != nullptr) skip[i].get(s);
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = (g[i][q] - xh[i][q] * dot) * rstd + s[q];
      if (lane + i * lanes < chunks) store_rounded<kType>(a.grad_x, row + (lane + i * lanes) * 8, f);
    }
  }
  if (a.grad_weight == nullptr) return;
  float* part = a.partial + static_cast<int64_t>(blockIdx.x) * a.hidden;
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
    if (lane + i * lanes < chunks) store_rounded<Out::kF32>(part, (lane + i * lanes) * 8, dw[i]);
}

// Sums the parts: a workgroup has 64 columns, a wave every kSumWaves-th part of
// them, and the waves' sums are added in order.
constexpr int kSumWaves = 8;
__global__ __launch_bounds__(kWave* kSumWaves) void rms_norm_weight_sum_kernel(const float* partial, int32_t parts,
                                                                              int32_t hidden, float* grad_weight) {
  __shared__ float lds[kSumWaves][kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int col = blockIdx.x * kWave + lane;
  float s = 0.0f;
  if (col < hidden)
    for (int p = wave; p < parts; p += kSumWaves) s += partial[static_cast<int64_t>(p) * hidden + col];
  lds[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || col >= hidden) return;
#pragma unroll
  for (int q = 1; q < kSumWaves; ++q) s += lds[q][lane];
  grad_weight[col] = s;
}

// f(chunks, one wave) with the shape as compile-time constants.
template <typename F>
hipError_t with_norm_shape(select::NormShape s, F f) {
  const auto chunks = [&](auto one) {
    switch (s.chunks) {
      case 1: return f(std::integral_constant<int, 1>{}, one);
      case 2: return f(std::integral_constant<int, 2>{}, one);
      case 4: return f(std::integral_constant<int, 4>{}, one);
    }
    return hipErrorInvalidValue;
  };
  return s.waves == 1 ? chunks(std::true_type{}) : chunks(std::false_type{});
}

template <Out kType>
hipError_t launch_norm_type(const NormArgs& a, hipStream_t stream) {
  const select::NormShape s = select::norm_shape(a.bs, a.hidden);
  return with_norm_shape(s, [&](auto chunks, auto one) {
    constexpr int kRows = decltype(one)::value ? select::kNormRowsPerGroup : 1;
    rms_norm_kernel<kType, decltype(chunks)::value, decltype(one)::value>
        <<<dim3((a.bs + kRows - 1) / kRows), dim3(kWave * (kRows > 1 ? kRows : s.waves)), 0, stream>>>(a);
    return hipGetLastError();
  });
}

template <Out kType, Out kGrad>
hipError_t launch_backward_types(const NormBackwardArgs& a, hipStream_t stream) {
  const select::NormShape s = select::norm_backward_shape(a.bs, a.hidden);
  const int32_t parts = select::norm_backward_parts(a.bs);
  const hipError_t e = a.bs == 0 ? hipSuccess : with_norm_shape(s, [&](auto chunks, auto one) {
    rms_norm_backward_kernel<kType, kGrad, decltype(chunks)::value, decltype(one)::value>
        <<<dim3(parts), dim3(kWave * s.waves), 0, stream>>>(a);
    return hipGetLastError();
  });
  if (e != hipSuccess || a.grad_weight == nullptr) return e;
  rms_norm_weight_sum_kernel<<<dim3((a.hidden + kWave - 1) / kWave), dim3(kWave * kSumWaves), 0, stream>>>(
      a.partial, parts, a.hidden, a.grad_weight);
  return hipGetLastError();
}

template <Out kType>
hipError_t launch_backward_type(const NormBackwardArgs& a, Out grad_type, hipStream_t stream) {
  switch (grad_type) {
    case Out::kBf16: return launch_backward_types<kType, Out::kBf16>(a, stream);
    case Out::kFp16: return launch_backward_types<kType, Out::kFp16>(a, stream);
    case Out::kF32: return launch_backward_types<kType, Out::kF32>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, Out type, hipStream_t stream) {
  const int64_t size = type == Out::kF32 ? 4 : 2, out_size = a.out_type == Out::kF32 ? 4 : 2;
  for (int64_t first = 0; first < a.bs; first += select::kNormLaunchRows) {
    NormArgs p = a;
    const int64_t at = first * a.hidden;
    p.bs = static_cast<int32_t>(a.bs - first < select::kNormLaunchRows ? a.bs - first : select::kNormLaunchRows);
    p.x = static_cast<const uint8_t*>(a.x) + at * size;
    if (a.residual != nullptr) p.residual = static_cast<const uint8_t*>(a.residual) + at * size;
    if (a.sum != nullptr) p.sum = static_cast<uint8_t*>(a.sum) + at * size;
    if (a.out != nullptr) p.out = static_cast<uint8_t*>(a.out) + at * out_size;
    if (a.rows != nullptr) p.rows = a.rows + first * a.row_bytes;
    if (a.rstd != nullptr) p.rstd = a.rstd + first;
    hipError_t e = hipErrorInvalidValue;
    switch (type) {
      case Out::kBf16: e = launch_norm_type<Out::kBf16>(p, stream); break;
      case Out::kFp16: e = launch_norm_type<Out::kFp16>(p, stream); break;
      case Out::kF32: e = launch_norm_type<Out::kF32>(p, stream); break;
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_rms_norm_backward(const NormBackwardArgs& a, Out type, Out grad_type, hipStream_t stream) {
  switch (type) {
    case Out::kBf16: return launch_backward_type<Out::kBf16>(a, grad_type, stream);
    case Out::kFp16: return launch_backward_type<Out::kFp16>(a, grad_type, stream);
    case Out::kF32: return launch_backward_type<Out::kF32>(a, grad_type, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
