// The router: each token's topk experts and their weights from its logits.
//
// A token is the work of 16 lanes (four tokens a wave; up to 256 experts and
// 16 entries, batches that fill the chip that way) or of a wave; lane l holds
// the kVpl experts from l kVpl.
//
// The choice is made on keys: binary64 whole numbers N 2^11 + (2047 - e),
// where N orders the selection values of the experts -- the grid value u 2^30
// of a biased score (|u| <= 2^10, so |N| <= 2^40, and 2^41 for a sum of two),
// or the logit's bits mapped to a whole number of the same order -- and the
// expert's id e below it settles ties for the lower id.  Every key is exact
// (at most 2^52 + 2^11) and no two are equal, so one maximum (a v_max_f64 takes
// as long as a v_max_f32 here) names value and expert at once.  A lane sorts
// its keys; then each of k rounds takes the largest of the lanes' first keys,
// and the lane that had it moves its list up.  Groups are ranked by the same
// means.
//
// Scores for the choice are computed in binary64 (exp64 below; the error of a
// score is below 2^-44, far below the grid), weights in binary32.
#include "device_util.h"
#include "launch.h"
#include "router_util.h"

namespace moe {
namespace {

constexpr int kWaves = 4;
constexpr double kNone = -__builtin_inf();  // the key of an expert that cannot be chosen
constexpr int kIdBits = 11;
constexpr double kIdSpan = 1 << kIdBits;
static_assert(MOE_MAX_EXPERTS <= (1 << kIdBits) && MOE_ROUTE_MAX_GROUPS <= kWave, "ids fit below the value");

__device__ __forceinline__ double make_key(double value, int id) {
  return __builtin_fma(value, kIdSpan, static_cast<double>((1 << kIdBits) - 1 - id));  // exact
}
// The id below a key: what is left of the key past whole multiples of 2^11
// (every step exact, also for the sum of two values at their bound).
__device__ __forceinline__ int key_id(double key) {
  const double below = __builtin_fma(__builtin_floor(key * (1.0 / kIdSpan)), -kIdSpan, key);
  return (1 << kIdBits) - 1 - static_cast<int>(below);
}

// Whole number of the same order as the (finite) logit.
__device__ __forceinline__ double logit_value(float x) {
  const int b = __float_as_int(x);
  return static_cast<double>(b ^ ((b >> 31) & 0x7fffffff));
}

// e^x for |x| <= 64: x = n ln 2 + r, |r| <= ln(2) / 2, the Taylor polynomial
// of degree 11 (its remainder is below r^12 / 12! e^r < 2^-46 of the result),
// times 2^n.
__device__ __forceinline__ double exp64(double x) {
  const double n = __builtin_rint(x * 1.4426950408889634);
  const double r = __builtin_fma(n, -0.6931471805599453, x);
  double p = 1.0 / 39916800.0;
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, static_cast<int>(n));
}
// 1 / d for 1 <= d: the hardware's estimate and two Newton steps.
__device__ __forceinline__ double reciprocal(double d) {
  double y = __builtin_amdgcn_rcp(d);
  y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
  return __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
}

// Descending sort of kN (a power of two) keys: Batcher's odd-even merge sort.
template <int kN>
__device__ __forceinline__ void sort_keys(double (&v)[kN]) {
#pragma unroll
  for (int p = 1; p < kN; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < kN; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < kN && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const double a = v[i + j], b = v[i + j + q];
            v[i + j] = __builtin_fmax(a, b);
            v[i + j + q] = __builtin_fmin(a, b);
          }
}

// Whether a group is whole lanes, 1, 2, 4, 8 or 16 of them.
constexpr bool lane_groups(int group_size, int vpl) {
  const int lanes = group_size / vpl;
  return group_size % vpl == 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0;
}

template <bool kSigmoid, int kL, int kVpl>
__global__ __launch_bounds__(kWaves* kWave) void route_kernel(RouterArgs a, Out type) {
  extern __shared__ __attribute__((aligned(16))) double lds[];  // [tokens][E], if groups are not whole lanes
  constexpr int kTokens = kWave / kL;
  const int lane = threadIdx.x % kL, sub = threadIdx.x / kL;  // lane of the token, token of the workgroup
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (kTokens * kWaves) + sub;
  const bool active = token < a.bs;
  const int64_t t = active ? token : a.bs - 1;  // lanes past the batch work on its last token and store nothing
  const int e0 = lane * kVpl;
  const bool masked = a.token_mask != nullptr && a.token_mask[t] == 0;

  float x[kVpl];
  load_logits<kVpl>(a.logits, type, t * a.stride + e0, a.num_experts - e0, x);
  if (masked) {
#pragma unroll
    for (int i = 0; i < kVpl; ++i) x[i] = -__builtin_inff();
  }

  // the whole row's softmax statistics, where the scores need them
  const bool scored = a.bias != nullptr || (a.groups > 1 && a.group_top == 2);
  float top = 0.0f, sum = 1.0f;
  if (!kSigmoid && (scored || !a.renorm)) {
    top = x[0];
#pragma unroll
    for (int i = 1; i < kVpl; ++i) top = __builtin_fmaxf(top, x[i]);
    top = token_max<kL>(top);
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kVpl; ++i) sum += x[i] > -__builtin_inff() ? expf(x[i] - top) : 0.0f;
    sum = token_sum<kL>(sum);
  }

  double v[kVpl];  // selection values as whole numbers, then keys
#pragma unroll
  for (int i = 0; i < kVpl; ++i) v[i] = x[i] > -__builtin_inff() ? logit_value(x[i]) : kNone;
  double best2 = kNone, best1 = kNone;  // the largest values of this lane's experts, for their group
  if (scored) {
    double u[kVpl], z = 0.0;
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      const bool ok = x[i] > -__builtin_inff();
      if constexpr (kSigmoid) {
        const float c = __builtin_amdgcn_fmed3f(ok ? x[i] : 0.0f, -64.0f, 64.0f);  // past that s is 0 or 1 on the grid
        u[i] = reciprocal(1.0 + exp64(-static_cast<double>(c)));
      } else {
        const double d = ok ? static_cast<double>(x[i]) - static_cast<double>(top) : 0.0;
        u[i] = ok ? exp64(__builtin_fmax(d, -64.0)) : 0.0;
        z += u[i];
      }
    }
    const double share = kSigmoid ? 1.0 : reciprocal(__builtin_fmax(token_sum<kL>(z), 1.0));
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      double s = kSigmoid ? u[i] : u[i] * share;
      if (a.bias != nullptr) s += static_cast<double>(a.bias[min(e0 + i, a.num_experts - 1)]);
      u[i] = v[i] > kNone ? __builtin_rint(__builtin_fmin(__builtin_fmax(s, -1024.0), 1024.0) * 1073741824.0) : kNone;
      if (a.bias != nullptr) v[i] = u[i];
      best2 = __builtin_fmax(best2, __builtin_fmin(best1, u[i]));
      best1 = __builtin_fmax(best1, u[i]);
    }
    if (a.groups > 1 && a.group_top == 2 && !lane_groups(a.group_size, kVpl)) {
#pragma unroll
      for (int i = 0; i < kVpl; ++i)
        if (e0 + i < a.num_experts) lds[sub * a.num_experts + e0 + i] = u[i];
    }
  }

  if (a.groups > 1) {
    if (a.group_top == 1) {
      best1 = v[0];
#pragma unroll
      for (int i = 1; i < kVpl; ++i) best1 = __builtin_fmax(best1, v[i]);
    }
    uint64_t kept = 0;
    if (lane_groups(a.group_size, kVpl)) {
      const int lanes = a.group_size / kVpl;
      // best1, best2 over the group's lanes: of two lanes' pairs, the two largest
      const auto merge = [&](double o1, double o2) {
        best2 = __builtin_fmax(__builtin_fmax(best2, o2), __builtin_fmin(best1, o1));
        best1 = __builtin_fmax(best1, o1);
      };
      if (lanes > 1) merge(dpp<kDppXor1>(best1), dpp<kDppXor1>(best2));
      if (lanes > 2) merge(dpp<kDppXor2>(best1), dpp<kDppXor2>(best2));
      if (lanes > 4) merge(dpp<kDppMirror8>(best1), dpp<kDppMirror8>(best2));
      if (lanes > 8) merge(dpp<kDppMirror16>(best1), dpp<kDppMirror16>(best2));
      const int g = lane / lanes;
      if (a.group_top == 2 && best2 > kNone) best1 += best2;
      double key = g < a.groups && best1 > kNone ? make_key(best1, g) : kNone;
      bool keep = false;
      for (int j = 0; j < a.keep; ++j) {
        const double best = token_max<kL>(key);
        if (key == best) keep = true, key = kNone;  // all of its lanes (or none is left)
      }
#pragma unroll
      for (int i = 0; i < kVpl; ++i)
        if (!keep) v[i] = kNone;
    } else {
      double* values = lds + sub * a.num_experts;
      if (a.group_top == 1) {
#pragma unroll
        for (int i = 0; i < kVpl; ++i)
          if (e0 + i < a.num_experts) values[e0 + i] = v[i];
      }
      wave_lds_sync();
      constexpr int kRounds = MOE_ROUTE_MAX_GROUPS / kL;
      double key[kRounds];
#pragma unroll
      for (int r = 0; r < kRounds; ++r) {
        const int g = r * kL + lane;
        double first = kNone, second = kNone;
        if (g < a.groups) {
          for (int m = 0; m < a.group_size; ++m) {
            const double q = values[g * a.group_size + m];
            second = __builtin_fmax(second, __builtin_fmin(first, q));
            first = __builtin_fmax(first, q);
          }
        }
        if (a.group_top == 2 && second > kNone) first += second;
        key[r] = first > kNone ? make_key(first, g) : kNone;
      }
      for (int j = 0; j < a.keep; ++j) {
        double best = key[0];
#pragma unroll
        for (int r = 1; r < kRounds; ++r) best = __builtin_fmax(best, key[r]);
        best = token_max<kL>(best);
        if (best > kNone) kept |= uint64_t(1) << key_id(best);
#pragma unroll
        for (int r = 0; r < kRounds; ++r)
          if (key[r] == best) key[r] = kNone;
      }
#pragma unroll
      for (int i = 0; i < kVpl; ++i) {
        const int g = static_cast<int>((static_cast<uint64_t>(e0 + i) * a.group_magic) >> 32);
        if (!((kept >> (g & 63)) & 1)) v[i] = kNone;
      }
    }
  }

#pragma unroll
  for (int i = 0; i < kVpl; ++i)
    if (v[i] > kNone) v[i] = make_key(v[i], e0 + i);
  sort_keys<kVpl>(v);
  double mine = kNone;  // lane j: the key of entry j
  for (int j = 0; j < a.k; ++j) {
    const double best = token_max<kL>(v[0]);
    if (lane == j) mine = best;
    if (v[0] == best) {
#pragma unroll
      for (int i = 0; i + 1 < kVpl; ++i) v[i] = v[i + 1];
      v[kVpl - 1] = kNone;
    }
  }
  const int id = mine > kNone ? key_id(mine) : -1;

  const float xm = id >= 0 ? router_logit(load_logit(a.logits, type, t * a.stride + id)) : -__builtin_inff();
  float w = 0.0f;
  if (a.renorm) {
    const float m = token_max<kL>(xm);
    const float r = id >= 0 ? relative_score<kSigmoid>(xm, m) : 0.0f;
    const float z = token_sum<kL>(r);
    if (id >= 0) w = r / z;
  } else if (id >= 0) {
    w = kSigmoid ? sigmoid_f32(xm) : expf(xm - top) / sum;
  }
  if (active && lane < a.k) {
    const int64_t o = token * a.k + lane;
    a.topk_idx[o] = id;
    a.topk_weights[o] = w * a.scale;
  }
}

template <bool kSigmoid, int kL, int kVpl>
hipError_t launch_shape(const RouterArgs& a, Out type, hipStream_t stream) {
  constexpr int kTokens = kWave / kL * kWaves;
  const dim3 grid(static_cast<unsigned>((a.bs + kTokens - 1) / kTokens)), block(kWaves * kWave);
  // at most 16 tokens x 256 experts or 4 x 2048, 64 KB
  const size_t lds = a.groups > 1 && !lane_groups(a.group_size, kVpl) ? sizeof(double) * kTokens * a.num_experts : 0;
  hipLaunchKernelGGL((route_kernel<kSigmoid, kL, kVpl>), grid, block, lds, stream, a, type);
  return hipGetLastError();
}

// One case per entry of select::kRouterShapes.
template <bool kSigmoid>
hipError_t launch_score(const RouterArgs& a, Out type, hipStream_t stream) {
  const select::RouterShape s = select::router_shape(a.bs, a.num_experts, a.k);
#define MOE_ROUTE_CASE(L, V) \
  if (s.lanes == (L) && s.vpl == (V)) return launch_shape<kSigmoid, L, V>(a, type, stream);
  MOE_ROUTE_CASE(16, 1)
  MOE_ROUTE_CASE(16, 2)
  MOE_ROUTE_CASE(16, 4)
  MOE_ROUTE_CASE(16, 8)
  MOE_ROUTE_CASE(16, 16)
  MOE_ROUTE_CASE(64, 1)
  MOE_ROUTE_CASE(64, 2)
  MOE_ROUTE_CASE(64, 4)
  MOE_ROUTE_CASE(64, 8)
  MOE_ROUTE_CASE(64, 16)
  MOE_ROUTE_CASE(64, 32)
#undef MOE_ROUTE_CASE
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_route(const RouterArgs& a, Out logits_type, bool sigmoid, hipStream_t stream) {
  return sigmoid ? launch_score<true>(a, logits_type, stream) : launch_score<false>(a, logits_type, stream);
}

}  // namespace moe
