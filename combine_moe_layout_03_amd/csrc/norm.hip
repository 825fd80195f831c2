// Root-mean-square norm with the residual's addition, in front of the router
// and the dispatch, and its gradient.  For a row x of a token
//   s = round(x + residual), rstd = 1 / sqrt(mean(s^2) + eps), y = (s rstd) w
//   out = round(y), and 8-bit rows of y (block_rows.h)
// Sums are binary32: a lane's chunks in order, then the lanes, then the waves.
//
// A row's chunks of 8 elements lie in the registers of its lanes from the load
// to the stores, so every element is read and written once.  16 neighbouring
// lanes hold the 128 columns of an 8-bit block.
//
// Bound by the rows' bytes.  4096 tokens, h 7168, bf16, with the sum, the result
// and the 8-bit rows written: 47.2 us for 265 MB = 5.6 TB/s (43.0 at the fastest
// copy's 6.17).  The gradient of the same tokens, 235 MB: 43.0 us and 4.7 for
// the weight's parts (38.1).  A row stays in one workgroup, since its mean is
// needed before its first store; what hides a row's two barriers is the other
// rows of the CU, and in the gradient, whose workgroups walk many rows, the next
// row's loads.
#include "block_rows.h"
#include "device_util.h"
#include "norm.h"
#include "router_util.h"

#pragma clang fp contract(off)

namespace moe {
namespace {

constexpr int kMaxWaves = 8;  // of a workgroup (select::norm_shape keeps to it)
static_assert(select::norm_shape(MOE_MAX_HIDDEN).waves <= kMaxWaves && select::norm_shape(8192).waves <= kMaxWaves);

// Eight elements as they lie in memory.
template <Out kType>
struct Chunk {
  u32x4 w[kType == Out::kF32 ? 2 : 1];
  template <bool kNt>
  __device__ __forceinline__ void load(const void* base, int64_t elem) {
    const u32x4* p = reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(base) +
                                                    elem * (kType == Out::kF32 ? 4 : 2));
    w[0] = kNt ? __builtin_nontemporal_load(p) : p[0];
    if constexpr (kType == Out::kF32) w[1] = kNt ? __builtin_nontemporal_load(p + 1) : p[1];
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
  // Non-temporally: the rows read would else be pushed out of the caches by the
  // rows written.  The call gains, the kernel that reads the result next loses (h
  // 7168, bf16, us, non-temporally and not, in captured runs; the call, the call
  // and a router's product with 256 experts behind it, and copies of both results
  // in its place): 1 token 3.3, 3.3; 10.9, 11.0; 7.3, 6.8.  64: 3.7, 3.7; 14.5, 12.5;
  // 8.2, 8.2.  512: 6.8, 8.4; 24.1, 21.6; 18.1, 15.6.  2048: 26.5, 29.0; 52.8, 48.1;
  // 50.9, 46.0.  4096: 47.7, 45.2; 79.5, 72.3; 92.9, 93.0.  8192: 89.6, 99.1; 155,
  // 177; 184, 197.  The gradient and a copy of it: 512 17.0, 16.7; 2048 39.9, 37.7;
  // 4096 68.1, 64.6; 8192 123, 135.
  __device__ __forceinline__ void store(void* base, int64_t elem) const {
    u32x4* p = reinterpret_cast<u32x4*>(static_cast<uint8_t*>(base) + elem * (kType == Out::kF32 ? 4 : 2));
    __builtin_nontemporal_store(w[0], p);
    if constexpr (kType == Out::kF32) __builtin_nontemporal_store(w[1], p + 1);
  }
};

template <Out kType>
__device__ __forceinline__ void store_rounded(void* base, int64_t elem, float (&f)[8]) {
  Chunk<kType> c;
  c.round(f);
  c.store(base, elem);
}

// Eight floats where they are read again soon.
__device__ __forceinline__ void put_floats(float* to, const float (&f)[8]) {
  f32x4* p = reinterpret_cast<f32x4*>(to);
  p[0] = f32x4{f[0], f[1], f[2], f[3]};
  p[1] = f32x4{f[4], f[5], f[6], f[7]};
}

__device__ __forceinline__ void load_weight(const float* weight, int col, float (&w)[8]) {
  const f32x4_u* p = reinterpret_cast<const f32x4_u*>(weight + col);
  const f32x4 a = p[0], b = p[1];
#pragma unroll
  for (int q = 0; q < 4; ++q) w[q] = a[q], w[4 + q] = b[q];
}

// The sum of v over the row's waves, in every lane: of the workgroup's waves
// those from `first` on.
template <bool kOneWave>
__device__ __forceinline__ float row_sum(float v, int waves, float* lds, int first) {
  v = token_sum<kWave>(v);
  if constexpr (kOneWave) return v;
  if (threadIdx.x % kWave == 0) lds[threadIdx.x / kWave] = v;
  __syncthreads();
  float s = 0.0f;
  for (int q = 0; q < waves; ++q) s += lds[first + q];
  return s;
}

template <Out kType, int kChunks, bool kOneWave, bool kNt>
__global__ __launch_bounds__(kOneWave ? kWave* select::kNormRowsPerGroup : kWave* kMaxWaves) void rms_norm_kernel(
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
    x[i].template load<kNt>(a.x, row + c * 8);
    if (a.residual != nullptr) r[i].template load<kNt>(a.residual, row + c * 8);
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
  squares = row_sum<kOneWave>(squares, waves, lds, 0);
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
// A workgroup takes kRows rows at a time (as many as eight waves hold), and of
// the batch every parts-th such set.  A lane has the same columns of each row,
// so its part of dw stays in registers; the rows' parts are joined in LDS,
// written once, and summed by the second kernel, all in a fixed order.  The
// rows' chunks are loaded while the rows before them are summed (not where a
// lane has four chunks of each: the registers spill).
template <Out kType, Out kGrad, int kChunks, bool kOneWave, bool kNt>
__global__ __launch_bounds__(kWave* kMaxWaves) void rms_norm_backward_kernel(NormBackwardArgs a, int waves) {
  __shared__ float lds[2][kMaxWaves];
  __shared__ __attribute__((aligned(16))) float joined[select::kNormJoinedHidden];
  if constexpr (kOneWave) waves = 1;
  const int lanes = waves * kWave, rows = blockDim.x / lanes;
  const int lane = threadIdx.x % lanes, group = uniform(threadIdx.x / lanes);
  const int chunks = a.hidden / 8;
  float w[kChunks][8], dw[kChunks][8];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    load_weight(a.weight, min(lane + i * lanes, chunks - 1) * 8, w[i]);
#pragma unroll
    for (int q = 0; q < 8; ++q) dw[i][q] = 0.0f;
  }
  struct Row {
    Chunk<kGrad> g[kChunks];
    Chunk<kType> s[kChunks], skip[kChunks];
    float rstd;
    bool keep;
  };
  const auto load = [&](int64_t t, Row& r) {  // (past the batch its last row, which counts for nothing)
    t = t < a.bs ? t : a.bs - 1;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int64_t at = t * a.hidden + min(lane + i * lanes, chunks - 1) * 8;
      r.g[i].template load<kNt>(a.grad_out, at);
      r.s[i].template load<kNt>(a.sum, at);
      if (a.grad_sum != nullptr) r.skip[i].template load<kNt>(a.grad_sum, at);
    }
    r.rstd = a.rstd[t];
    r.keep = a.token_mask == nullptr || a.token_mask[t] != 0;  // the same in every lane of a row
  };
  const float mean = 1.0f / static_cast<float>(a.hidden);
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows;
  int turn = 0;
  Row next;
  if constexpr (kChunks <= 2) load(static_cast<int64_t>(blockIdx.x) * rows + group, next);
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * rows; first < a.bs; first += step) {
    const int64_t t = first + group;
    if constexpr (kChunks > 2) load(t, next);
    const Row now = next;
    if constexpr (kChunks <= 2) load(t + step, next);
    const bool counts = now.keep && t < a.bs;
    float g[kChunks][8], xh[kChunks][8], dot = 0.0f;
    if (counts) {
#pragma unroll
      for (int i = 0; i < kChunks; ++i) {
        now.g[i].get(g[i]);
        now.s[i].get(xh[i]);
        const bool mine = lane + i * lanes < chunks;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          xh[i][q] *= now.rstd;
          dw[i][q] = __builtin_fmaf(g[i][q], xh[i][q], dw[i][q]);
          g[i][q] *= w[i][q];
          if (mine) dot = __builtin_fmaf(g[i][q], xh[i][q], dot);
        }
      }
    }
    // the row's waves: `waves` of the workgroup's from group * waves on
    dot = row_sum<kOneWave>(dot, waves, lds[turn], group * waves) * mean;
    turn ^= 1;  // the other sums may still be read
    if (t >= a.bs) continue;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      float f[8], s[8] = {};
      if (a.grad_sum != nullptr) now.skip[i].get(s);
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = counts ? (g[i][q] - xh[i][q] * dot) * now.rstd + s[q] : 0.0f;
      if (lane + i * lanes < chunks) store_rounded<kType>(a.grad_x, t * a.hidden + (lane + i * lanes) * 8, f);
    }
  }
  if (a.grad_weight == nullptr) return;
  for (int r = 1; r < rows; ++r) {  // the first row's lanes add the others'
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if (group == r && lane + i * lanes < chunks) put_floats(joined + (lane + i * lanes) * 8, dw[i]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      if (group != 0 || lane + i * lanes >= chunks) continue;
#pragma unroll
      for (int q = 0; q < 8; ++q) dw[i][q] += joined[(lane + i * lanes) * 8 + q];
    }
  }
  if (group != 0) return;
  float* part = a.partial + static_cast<int64_t>(blockIdx.x) * a.hidden;
#pragma unroll
  for (int i = 0; i < kChunks; ++i)
    if (lane + i * lanes < chunks) put_floats(part + (lane + i * lanes) * 8, dw[i]);
}

// Sums the parts: a workgroup has 64 columns, a wave every kSumWaves-th part of
// them, kSumDeep loads at a time, and the waves' sums are added in order.
constexpr int kSumWaves = 16, kSumDeep = 8;
__global__ __launch_bounds__(kWave* kSumWaves) void rms_norm_weight_sum_kernel(const float* partial, int32_t parts,
                                                                              int32_t hidden, float* grad_weight) {
  __shared__ float lds[kSumWaves][kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int col = blockIdx.x * kWave + lane;
  const float* src = partial + min(col, hidden - 1);
  float s = 0.0f;
  for (int p0 = wave; p0 < parts; p0 += kSumWaves * kSumDeep) {
    float v[kSumDeep];
#pragma unroll
    for (int q = 0; q < kSumDeep; ++q) {
      const int p = p0 + q * kSumWaves;
      v[q] = src[static_cast<int64_t>(min(p, parts - 1)) * hidden];
      if (p >= parts) v[q] = 0.0f;
    }
#pragma unroll
    for (int q = 0; q < kSumDeep; ++q) s += v[q];
  }
  lds[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || col >= hidden) return;
#pragma unroll
  for (int q = 1; q < kSumWaves; ++q) s += lds[q][lane];
  grad_weight[col] = s;
}

// f(chunks, one wave, non-temporal loads) with the shape as compile-time
// constants.
template <int kChunks, bool kOneWave, bool kNt, typename F>
hipError_t call_shape(F f) {
  return f(std::integral_constant<int, kChunks>{}, std::bool_constant<kOneWave>{}, std::bool_constant<kNt>{});
}
template <typename F>
hipError_t with_norm_shape(select::NormShape s, bool nt, F f) {
  if (s.chunks == 1) return call_shape<1, true, false>(f);
  if (s.waves == 1) return call_shape<2, true, false>(f);
  if (s.chunks == 2) return nt ? call_shape<2, false, true>(f) : call_shape<2, false, false>(f);
  return nt ? call_shape<4, false, true>(f) : call_shape<4, false, false>(f);
}

template <Out kType>
hipError_t launch_norm_type(const NormArgs& a, hipStream_t stream) {
  const select::NormShape s = select::norm_shape(a.hidden);
  const int64_t read = static_cast<int64_t>(a.bs) * a.hidden * (kType == Out::kF32 ? 4 : 2) * (a.residual != nullptr ? 2 : 1);
  return with_norm_shape(s, select::norm_nt(read), [&](auto chunks, auto one, auto nt) {
    constexpr int kRows = decltype(one)::value ? select::kNormRowsPerGroup : 1;
    rms_norm_kernel<kType, decltype(chunks)::value, decltype(one)::value, decltype(nt)::value>
        <<<dim3((a.bs + kRows - 1) / kRows), dim3(kWave * (kRows > 1 ? kRows : s.waves)), 0, stream>>>(a);
    return hipGetLastError();
  });
}

template <Out kType, Out kGrad>
hipError_t launch_backward_types(const NormBackwardArgs& a, hipStream_t stream) {
  const select::NormShape s = select::norm_shape(a.hidden);
  const int32_t parts = select::norm_backward_parts(a.bs, a.hidden);
  const int64_t read = static_cast<int64_t>(a.bs) * a.hidden *
                       ((kType == Out::kF32 ? 4 : 2) * (a.grad_sum != nullptr ? 2 : 1) + (kGrad == Out::kF32 ? 4 : 2));
  const auto launch = [&](auto chunks, auto one, auto nt) {
    rms_norm_backward_kernel<kType, kGrad, decltype(chunks)::value, decltype(one)::value, decltype(nt)::value>
        <<<dim3(parts), dim3(kWave * s.waves * select::norm_backward_rows(s.waves)), 0, stream>>>(a, s.waves);
    return hipGetLastError();
  };
  const hipError_t e = a.bs == 0 ? hipSuccess : with_norm_shape(s, select::norm_nt(read), launch);
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
