// The router: each token's topk experts and their weights from its logits.
//
// One wave per token; lane l holds the logits of experts l + 64 i, i < kVpl.
// The choice is made on keys: binary64 whole numbers N 2^11 + (2047 - e),
// where N orders the selection values of the experts -- the grid value u 2^30
// of a biased score (|u| <= 2^10, so |N| <= 2^40, and 2^41 for a sum of two),
// or the logit's bits mapped to a whole number of the same order -- and the
// expert's id e below it settles ties for the lower id.  Every key is exact
// (at most 2^52 + 2^11) and no two are equal, so one maximum over the wave names value and expert at once; k
// of them, each followed by taking its expert out, give the choice in order.
// Groups are ranked by the same means.  Scores for the choice are computed in
// binary64, whose error is far below the grid.
#include "device_util.h"
#include "launch.h"
#include "router_util.h"

namespace moe {
namespace {

constexpr double kNone = -__builtin_inf();  // the key of an expert that cannot be chosen
constexpr int kIdBits = 11;
constexpr double kIdSpan = 1 << kIdBits;
static_assert(MOE_MAX_EXPERTS <= (1 << kIdBits) && MOE_ROUTE_MAX_GROUPS <= kWave, "ids fit below the value");

__device__ __forceinline__ double make_key(double value, int id) {
  return value * kIdSpan + static_cast<double>((1 << kIdBits) - 1 - id);
}
// The id below a key: what is left of the key past whole multiples of 2^11
// (every step exact, also for the sum of two values at their bound).
__device__ __forceinline__ int key_id(double key) {
  const double below = key - __builtin_floor(key * (1.0 / kIdSpan)) * kIdSpan;
  return (1 << kIdBits) - 1 - static_cast<int>(below);
}

// Whole number of the same order as the (finite) logit.
__device__ __forceinline__ double logit_value(float x) {
  const int b = __float_as_int(x);
  return static_cast<double>(b ^ ((b >> 31) & 0x7fffffff));
}

__device__ __forceinline__ double wave_max_f64(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v = __builtin_fmax(v, __shfl_xor(v, d, kWave));
  return v;
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

// Orders this wave's LDS writes before its later LDS reads of other lanes' data.
__device__ __forceinline__ void wave_lds_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

constexpr size_t route_lds_per_wave(int experts) { return static_cast<size_t>(experts) * 12u; }

template <Out kType, bool kSigmoid, int kVpl>
__global__ __launch_bounds__(256) void route_kernel(RouterArgs a) {
  extern __shared__ __attribute__((aligned(16))) double lds[];
  const int lane = threadIdx.x % kWave, wave = uniform(static_cast<int>(threadIdx.x / kWave));
  const int t = static_cast<int>(blockIdx.x) * static_cast<int>(blockDim.x / kWave) + wave;
  if (t >= a.bs) return;
  double* values = lds + static_cast<size_t>(wave) * a.num_experts;
  float* xs = reinterpret_cast<float*>(lds + static_cast<size_t>(blockDim.x / kWave) * a.num_experts) +
              static_cast<size_t>(wave) * a.num_experts;
  const bool masked = a.token_mask != nullptr && a.token_mask[t] == 0;

  float x[kVpl];
  bool ok[kVpl];
#pragma unroll
  for (int i = 0; i < kVpl; ++i) {
    const int e = lane + i * kWave;
    x[i] = -__builtin_inff();
    if (e < a.num_experts && !masked) x[i] = router_logit(load_float<kType>(a.logits, t * a.stride + e));
    ok[i] = x[i] > -__builtin_inff();
    if (e < a.num_experts) xs[e] = x[i];
  }

  // the whole row's softmax statistics, where the scores need them
  const bool scored = a.bias != nullptr || (a.groups > 1 && a.group_top == 2);
  float top = 0.0f, sum = 1.0f;
  if (!kSigmoid && (scored || !a.renorm)) {
    top = x[0];
#pragma unroll
    for (int i = 1; i < kVpl; ++i) top = __builtin_fmaxf(top, x[i]);
    top = wave_max_f32(top);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kVpl; ++i) sum += ok[i] ? expf(x[i] - top) : 0.0f;
    sum = wave_sum_f32(sum);
  }

  double v[kVpl];  // selection values as whole numbers
  double u[kVpl];
#pragma unroll
  for (int i = 0; i < kVpl; ++i) v[i] = u[i] = ok[i] ? logit_value(x[i]) : kNone;
  if (scored) {
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      const double d = static_cast<double>(x[i]);
      u[i] = !ok[i] ? 0.0 : kSigmoid ? 1.0 / (1.0 + exp(-d)) : exp(d - static_cast<double>(top));
      z += u[i];
    }
    if (!kSigmoid) z = wave_sum_f64(z);
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      const int e = lane + i * kWave;
      double s = kSigmoid ? u[i] : u[i] / z;
      if (a.bias != nullptr && e < a.num_experts) s += static_cast<double>(a.bias[e]);
      u[i] = ok[i] ? __builtin_rint(__builtin_fmin(__builtin_fmax(s, -1024.0), 1024.0) * 1073741824.0) : kNone;
      if (a.bias != nullptr) v[i] = u[i];
    }
  }

  if (a.groups > 1) {
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      const int e = lane + i * kWave;
      if (e < a.num_experts) values[e] = a.group_top == 2 ? u[i] : v[i];
    }
    wave_lds_sync();
    double first = kNone, second = kNone;
    if (lane < a.groups) {
      for (int m = 0; m < a.group_size; ++m) {
        const double q = values[lane * a.group_size + m];
        second = __builtin_fmax(second, __builtin_fmin(first, q));
        first = __builtin_fmax(first, q);
      }
    }
    if (a.group_top == 2 && second > kNone) first += second;
    double key = first > kNone ? make_key(first, lane) : kNone;
    uint64_t kept = 0;
    for (int j = 0; j < a.keep; ++j) {
      const double best = wave_max_f64(key);
      if (!(best > kNone)) break;
      kept |= uint64_t(1) << key_id(best);
      if (key == best) key = kNone;
    }
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      const int g = (lane + i * kWave) / a.group_size;
      if (!((kept >> (g & 63)) & 1)) v[i] = kNone;
    }
  }

#pragma unroll
  for (int i = 0; i < kVpl; ++i)
    if (v[i] > kNone) v[i] = make_key(v[i], lane + i * kWave);
  int mine = -1;  // lane j: the expert of entry j
  for (int j = 0; j < a.k; ++j) {
    double best = v[0];
#pragma unroll
    for (int i = 1; i < kVpl; ++i) best = __builtin_fmax(best, v[i]);
    best = wave_max_f64(best);
    if (!(best > kNone)) break;
    if (lane == j) mine = key_id(best);
#pragma unroll
    for (int i = 0; i < kVpl; ++i)
      if (v[i] == best) v[i] = kNone;
  }

  wave_lds_sync();
  const float xm = mine >= 0 ? xs[mine] : -__builtin_inff();
  float w = 0.0f;
  if (a.renorm) {
    const float m = wave_max_f32(xm);
    const float r = mine >= 0 ? relative_score<kSigmoid>(xm, m) : 0.0f;
    const float z = wave_sum_f32(r);
    if (mine >= 0) w = r / z;
  } else if (mine >= 0) {
    w = kSigmoid ? sigmoid_f32(xm) : expf(xm - top) / sum;
  }
  if (lane < a.k) {
    const int64_t o = static_cast<int64_t>(t) * a.k + lane;
    a.topk_idx[o] = mine;
    a.topk_weights[o] = w * a.scale;
  }
}

template <Out kType, bool kSigmoid>
hipError_t launch_vpl(const RouterArgs& a, hipStream_t stream) {
  const int waves = a.num_experts <= 512 ? 4 : 1;  // LDS of a workgroup: at most 24 KB
  const dim3 grid(static_cast<unsigned>((a.bs + waves - 1) / waves)), block(static_cast<unsigned>(waves * kWave));
  const size_t lds = route_lds_per_wave(a.num_experts) * static_cast<size_t>(waves);
#define MOE_ROUTE_CASE(V)                                                                  \
  case V:                                                                                  \
    hipLaunchKernelGGL((route_kernel<kType, kSigmoid, V>), grid, block, lds, stream, a);   \
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

hipError_t launch_route(const RouterArgs& a, Out logits_type, bool sigmoid, hipStream_t stream) {
  switch (logits_type) {
    case Out::kBf16: return launch_score<Out::kBf16>(a, sigmoid, stream);
    case Out::kFp16: return launch_score<Out::kFp16>(a, sigmoid, stream);
    case Out::kF32: return launch_score<Out::kF32>(a, sigmoid, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
