// The router: each token's topk experts and their weights from its logits.
//
// A token is the work of 16 lanes (four tokens a wave; up to 256 experts and
// 16 entries, batches that fill the chip that way) or of a wave; lane l holds
// the kVpl experts from l kVpl.
//
// The choice is made on keys: binary64 selection values -- score + bias, or the
// logit itself -- whose lowest 11 bits are replaced by the expert's id, so that
// of equal values the lower id has the larger key.  A value keeps 42 significant
// bits whatever its size (a logit has 24), and no two keys are equal, so one
// maximum (a v_max_f64 takes as long as a v_max_f32 here) names value and
// expert at once.  A lane sorts its keys; then each of k rounds takes the
// largest of the lanes' first keys, and the lane that had it moves its list up.
// Groups are ranked by the same means.  (Values on a grid of 2^-30 lost the
// order of scores that are all small, where binary32 scores keep it.)
//
// Scores for the choice are computed in binary64, off by less than 2^-40 of
// themselves (exp64.h: an exponential, for the softmax over a sum of such, and a
// reciprocal); weights in binary32.
//
// Bound by the vector ALU: some 1200 instructions for four tokens of 256
// experts, 450 of them the sigmoids (binary64 runs at the rate of binary32
// here), issued in 73 % of the cycles.  16384 tokens x 256 experts, 8 groups,
// fp32: 13 us, where the bytes alone take 2.9; 160 experts in 8 groups, which
// are not whole lanes: 17 us and 1.9.  A choice in 32 bits, with this one behind
// it for the waves in which values lie too close, was not faster (18 us: one
// token in 250 is such, and a launch waits for its slowest wave).
#include "device_util.h"
#include "exp64.h"
#include "layer.h"
#include "router_util.h"

namespace moe {
namespace {

// Waves of a workgroup: its tokens' LDS stays within 52 KB.
constexpr int route_waves(int lanes, int vpl) { return lanes * vpl > 512 ? 2 : 4; }
// The value and the key of an expert that cannot be chosen: any number below
// kNone (see unless()), which is below every logit.
constexpr double kNone = -1e200;
constexpr uint32_t kIdMask = 2047;  // the bits of a key that hold the id
static_assert(MOE_MAX_EXPERTS <= kIdMask + 1 && MOE_ROUTE_MAX_GROUPS <= kWave, "ids fit below the value");

// v, or if `none` a number below kNone: one select, of the upper word.
__device__ __forceinline__ double unless(bool none, double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint64_t hi = none ? uint64_t(0xf8300000) : b >> 32;  // about -2^900
  return __builtin_bit_cast(double, (hi << 32) | (b & 0xffffffffu));
}

// The id's bits count down for a positive value and up for a negative one: of
// two keys of one value the lower id's is the larger.  `not_id` is ~id in the
// bits of kIdMask.
__device__ __forceinline__ double make_key(double value, uint32_t not_id) {
  const uint64_t b = __builtin_bit_cast(uint64_t, value);
  const uint32_t hi = static_cast<uint32_t>(b >> 32), sign = static_cast<uint32_t>(static_cast<int32_t>(hi) >> 31);
  uint32_t lo;  // (the compiler takes five instructions for these three)
  asm("v_bfi_b32 %0, %1, %2, %3" : "=v"(lo) : "s"(kIdMask), "v"(not_id ^ sign), "v"(static_cast<uint32_t>(b)));
  return __builtin_bit_cast(double, (uint64_t(hi) << 32) | lo);
}
// A key's value, and any value as a key holds it; a key's id.
__device__ __forceinline__ double key_value(double key) {
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, key) & ~uint64_t(kIdMask));
}
__device__ __forceinline__ int key_id(double key) {
  const uint64_t b = __builtin_bit_cast(uint64_t, key);
  const uint32_t sign = static_cast<uint32_t>(static_cast<int32_t>(b >> 32) >> 31);
  return static_cast<int>((~static_cast<uint32_t>(b) ^ sign) & kIdMask);
}

// e^x (exp64.h).  The coefficients are kept out of the compiler's sight: for ones
// that it knows, each v_fmac_f64 gets two moves.
struct Exp64 {
  double c[8];
  __device__ __forceinline__ Exp64() {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = kExpTerms[i];
      asm("" : "+v"(c[i]));
    }
  }
  __device__ __forceinline__ double operator()(double x) const {
    const double n = __builtin_rint(x * kLog2E);
    return __builtin_amdgcn_ldexp(exp_reduced(c, x, n), static_cast<int>(n));
  }
};
// 1 / d for 1 <= d: the hardware's estimate (2^-24) and a Newton step.
__device__ __forceinline__ double reciprocal(double d) {
  const double y = __builtin_amdgcn_rcp(d);
  return __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
}

__device__ __forceinline__ double larger(double a, double b) { return __builtin_fmax(a, b); }
__device__ __forceinline__ double smaller(double a, double b) { return __builtin_fmin(a, b); }

// Descending sort of kN (a power of two) keys from v[kAt]: Batcher's odd-even
// merge sort.
template <int kN, int kAt, int kAll>
__device__ __forceinline__ void sort_keys(double (&v)[kAll]) {
#pragma unroll
  for (int p = 1; p < kN; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < kN; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < kN && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const double a = v[kAt + i + j], b = v[kAt + i + j + q];
            v[kAt + i + j] = larger(a, b);
            v[kAt + i + j + q] = smaller(a, b);
          }
}

// w, sorted descending, becomes the 8 largest keys of itself and `other`, also
// sorted: the larger ones of the first list and the reversed second are those,
// as a bitonic sequence that three rounds sort.
template <int kAll, typename Other>
__device__ __forceinline__ void join8(double (&w)[kAll], Other other) {
  double h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = larger(w[i], other(7 - i));
#pragma unroll
  for (int d = 4; d >= 1; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & d) == 0) {
        const double p = h[i], q = h[i + d];
        h[i] = larger(p, q);
        h[i + d] = smaller(p, q);
      }
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = h[i];
}

// Whether a choice takes lists of 8: every entry may come from one lane.
template <int kL, int kVpl>
__device__ __forceinline__ bool lists_of_8(int k) {
  return kL == 16 && kVpl >= 8 && k <= 8;
}

// A lane's keys in descending order (its 8 largest, for lists of 8).
template <int kL, int kVpl>
__device__ __forceinline__ void sort_lane(double (&v)[kVpl], int k) {
  if constexpr (kL == 16 && kVpl == 16) {
    if (lists_of_8<kL, kVpl>(k)) {
      sort_keys<8, 0>(v);
      sort_keys<8, 8>(v);
      double w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = v[8 + i];
      join8(v, [&](int i) { return w[i]; });
      return;
    }
  }
  sort_keys<kVpl, 0>(v);
}

// Whether a group is whole lanes, 1, 2, 4, 8 or 16 of them.
constexpr bool lane_groups(int group_size, int vpl) {
  const int lanes = group_size / vpl;
  return group_size % vpl == 0 && lanes <= 16 && (lanes & (lanes - 1)) == 0;
}

// The selection values of a lane's experts: their scores with the bias.
template <bool kSigmoid, int kL, int kVpl>
__device__ __forceinline__ void score_values(const float (&x)[kVpl], const float (&bias)[kVpl], float top,
                                             double (&u)[kVpl]) {
  constexpr double kClip = 1024.0;
  const Exp64 exp64;
  if constexpr (kSigmoid) {
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      // binary32 has no score below e^-104, and they are equal here
      const float c = __builtin_amdgcn_fmed3f(x[i], -104.0f, 104.0f);
      u[i] = reciprocal(1.0 + exp64(-static_cast<double>(c))) + static_cast<double>(bias[i]);
    }
  } else {
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      // (times a share of 2^-11 or more that is still a normal number)
      u[i] = exp64(__builtin_fmax(static_cast<double>(x[i]) - static_cast<double>(top), -690.0));
      z += x[i] > -__builtin_inff() ? u[i] : 0.0;
    }
    const double share = reciprocal(__builtin_fmax(token_sum<kL>(z), 1.0));
#pragma unroll
    for (int i = 0; i < kVpl; ++i) u[i] = __builtin_fma(u[i], share, static_cast<double>(bias[i]));
  }
  float size = 0.0f;
#pragma unroll
  for (int i = 0; i < kVpl; ++i) size += __builtin_fabsf(bias[i]);
  if (__any(!(size <= 1000.0f))) {  // some may be large, infinite or NaN
    asm volatile("");  // a branch, not selects
#pragma unroll
    for (int i = 0; i < kVpl; ++i)
      u[i] = unless(!(bias[i] > -__builtin_inff()), __builtin_fmin(__builtin_fmax(u[i], -kClip), kClip));
  }
#pragma unroll
  for (int i = 0; i < kVpl; ++i) u[i] = unless(!(x[i] > -__builtin_inff()), u[i]);
}

// A group's two largest values, over lanes with merge().
struct TwoLargest {
  double first = 2 * kNone, second = 2 * kNone;
  __device__ __forceinline__ void add(double q) {
    second = __builtin_fmax(second, __builtin_fmin(first, q));
    first = __builtin_fmax(first, q);
  }
  template <int kCtrl>
  __device__ __forceinline__ void merge() {
    const double o1 = dpp<kCtrl>(first), o2 = dpp<kCtrl>(second);
    second = __builtin_fmax(__builtin_fmax(second, o2), __builtin_fmin(first, o1));
    first = __builtin_fmax(first, o1);
  }
  // Over 2^lanes_log2 lanes side by side.
  __device__ __forceinline__ void merge_lanes(int lanes_log2) {
    if (lanes_log2 > 0) merge<kDppXor1>();
    if (lanes_log2 > 1) merge<kDppXor2>();
    if (lanes_log2 > 2) merge<kDppMirror8>();
    if (lanes_log2 > 3) merge<kDppMirror16>();
  }
  // The group's value; below kNone where it has no eligible expert.
  __device__ __forceinline__ double value(int group_top) const {
    return group_top == 2 && second > kNone ? first + second : first;
  }
};

// Whether this lane's group is one of the best, for groups of whole lanes;
// `best`: the lane's own two largest values.
template <int kL, int kVpl>
__device__ __forceinline__ bool keep_lane(const RouterArgs& a, TwoLargest best, int lane) {
  const int lanes_log2 = __builtin_ctz(a.group_size / kVpl);
  best.merge_lanes(lanes_log2);
  double key = make_key(best.value(a.group_top), ~static_cast<uint32_t>(lane >> lanes_log2));
  bool keep = false;
  for (int j = 0; j < a.keep; ++j)
    if (key == token_max<kL>(key)) keep = true, key = 2 * kNone;  // all of the group's lanes
  return keep;
}

// Place of an expert's value: a lane's experts apart from the next lane's by
// one, so that lanes that store together meet in few banks (16384 tokens, 160
// experts, 8 groups: 15.1 us instead of 16.8 when this was measured, 16.5 with
// the keys of now; with fewer experts a lane the places cost what the banks did).
template <int kVpl>
__device__ __forceinline__ int value_place(int e) {
  return kVpl >= 16 ? e + e / kVpl : e;
}

// The groups that are kept, as bits, for groups of any size; `values`: LDS with
// the values of the token's experts.  Few groups get up to 16 lanes each (2
// tokens, 352 experts, 2 groups: 5.9 us instead of 9.7 with a lane each).
template <int kL, int kVpl>
__device__ __forceinline__ uint64_t keep_bits(const RouterArgs& a, int lane, const double* values) {
  constexpr int kRounds = MOE_ROUTE_MAX_GROUPS / kL;
  int share = 0;  // log2 of a group's lanes
  while (share < 4 && a.groups << (share + 1) <= kL) ++share;
  double key[kRounds];
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int g = r * kL + (lane >> share);
    TwoLargest best;
    if (g < a.groups)
      for (int m = lane & ((1 << share) - 1); m < a.group_size; m += 1 << share)
        best.add(values[value_place<kVpl>(g * a.group_size + m)]);
    if (r == 0) best.merge_lanes(share);  // more rounds are of groups with a lane each
    key[r] = make_key(best.value(a.group_top), ~static_cast<uint32_t>(g));
  }
  uint64_t kept = 0;
  for (int j = 0; j < a.keep; ++j) {
    double best = key[0];
#pragma unroll
    for (int r = 1; r < kRounds; ++r) best = __builtin_fmax(best, key[r]);
    best = token_max<kL>(best);
    if (best > kNone) kept |= uint64_t(1) << key_id(best);
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
      if (key[r] == best) key[r] = 2 * kNone;
  }
  return kept;
}

// Lane j's result is the j-th largest key of the token's lanes (j < k); v is
// sorted.
template <int kL, int kVpl>
__device__ __forceinline__ double largest_keys(double (&v)[kVpl], int k, int lane) {
  double mine = 2 * kNone;
  if constexpr (kL == 16 && kVpl >= 8) {
    if (lists_of_8<kL, kVpl>(k)) {
      // After four exchanges every lane has the token's 8 largest keys (some
      // 240 instructions; the loop below takes 45 a round).
      double w[8];
      const auto join = [&](auto other) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = v[i];
        join8(v, [&](int i) { return other(w[i]); });
      };
      join([](double q) { return dpp<kDppXor1>(q); });
      join([](double q) { return dpp<kDppXor2>(q); });
      join([](double q) { return dpp<kDppMirror8>(q); });
      join([](double q) { return dpp<kDppMirror16>(q); });
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (lane == i && i < k) mine = v[i];
      return mine;
    }
  }
  for (int j = 0; j < k; ++j) {
    const double best = token_max<kL>(v[0]);
    if (lane == j) mine = best;
    if (v[0] == best) {
#pragma unroll
      for (int i = 0; i + 1 < kVpl; ++i) v[i] = v[i + 1];
      v[kVpl - 1] = 2 * kNone;
    }
  }
  return mine;
}

template <bool kSigmoid, int kL, int kVpl>
__global__ __launch_bounds__(kWave* route_waves(kL, kVpl)) void route_kernel(RouterArgs a, Out type) {
  constexpr int kWaves = route_waves(kL, kVpl);
  extern __shared__ __attribute__((aligned(16))) double lds[];  // [tokens][E], if groups are not whole lanes
  constexpr int kTokens = kWave / kL;
  __shared__ __attribute__((aligned(16))) float logits[kWaves * kTokens][kL * kVpl];  // for the chosen ones
  const int lane = threadIdx.x % kL, sub = threadIdx.x / kL;  // lane of the token, token of the workgroup
  const int64_t token = static_cast<int64_t>(blockIdx.x) * (kTokens * kWaves) + sub;
  const bool active = token < a.bs;
  const int64_t t = active ? token : a.bs - 1;  // lanes past the batch work on its last token and store nothing
  const int e0 = lane * kVpl;
  double* values = lds + sub * value_place<kVpl>(a.num_experts);
  const bool masked = a.token_mask != nullptr && a.token_mask[t] == 0;

  float x[kVpl], bias[kVpl];
  load_logits<kVpl>(a.logits, type, t * a.stride + e0, a.num_experts - e0, x);
#pragma unroll
  for (int i = 0; i < kVpl; ++i) bias[i] = 0.0f;
  if (a.bias != nullptr) {
    if (kVpl % 4 == 0 && e0 + kVpl <= a.num_experts) {
#pragma unroll
      for (int i = 0; i < kVpl; i += 4) {
        const f32x4_u b = *reinterpret_cast<const f32x4_u*>(a.bias + e0 + i);
#pragma unroll
        for (int q = 0; q < 4; ++q) bias[i + q] = b[q];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVpl; ++i) bias[i] = a.bias[min(e0 + i, a.num_experts - 1)];
    }
  }
  if (masked) {
#pragma unroll
    for (int i = 0; i < kVpl; ++i) x[i] = -__builtin_inff();
  }
#pragma unroll
  for (int i = 0; i < kVpl; ++i) logits[sub][e0 + i] = x[i];

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

  double v[kVpl];  // selection values, then keys
  if (a.bias != nullptr) {
    score_values<kSigmoid, kL, kVpl>(x, bias, top, v);
  } else {
#pragma unroll
    for (int i = 0; i < kVpl; ++i) v[i] = unless(!(x[i] > -__builtin_inff()), static_cast<double>(x[i]));
  }
  // Groups are ranked by these values, or by scores of their own.  A lane of a
  // group of whole lanes sorts its keys first and has its group's candidates
  // on top of its list.
  const bool own_scores = a.groups > 1 && a.group_top == 2 && a.bias == nullptr;
  const bool whole_lanes = a.groups > 1 && lane_groups(a.group_size, kVpl);
  TwoLargest best;
  if (a.groups > 1 && (own_scores || !whole_lanes)) {
    double u[kVpl];
    if (own_scores) {
      score_values<kSigmoid, kL, kVpl>(x, bias, top, u);
    } else {
#pragma unroll
      for (int i = 0; i < kVpl; ++i) u[i] = v[i];
    }
#pragma unroll
    for (int i = 0; i < kVpl; ++i) u[i] = key_value(u[i]);
    if (whole_lanes) {
#pragma unroll
      for (int i = 0; i < kVpl; ++i) best.add(u[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kVpl; ++i)
        if (e0 + i < a.num_experts) values[value_place<kVpl>(e0) + i] = u[i];
      wave_lds_sync();
      const uint64_t kept = keep_bits<kL, kVpl>(a, lane, values);
#pragma unroll
      for (int i = 0; i < kVpl; ++i) {
        const int g = static_cast<int>((static_cast<uint64_t>(e0 + i) * a.group_magic) >> 32);
        v[i] = unless(!((kept >> (g & 63)) & 1), v[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kVpl; ++i) v[i] = make_key(v[i], ~static_cast<uint32_t>(e0) ^ static_cast<uint32_t>(i));
  sort_lane<kL, kVpl>(v, a.k);
  if (whole_lanes) {
    if (!own_scores) {
      best.first = key_value(v[0]);
      if constexpr (kVpl > 1) best.second = key_value(v[1]);
    }
    const bool keep = keep_lane<kL, kVpl>(a, best, lane);
#pragma unroll
    for (int i = 0; i < kVpl; ++i) v[i] = unless(!keep, v[i]);
  }
  const double mine = largest_keys<kL, kVpl>(v, a.k, lane);
  const int id = mine > kNone ? key_id(mine) : -1;

  wave_lds_sync();
  const float xm = id >= 0 ? logits[sub][id] : -__builtin_inff();
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
  constexpr int kWaves = route_waves(kL, kVpl), kTokens = kWave / kL * kWaves;
  const dim3 grid(static_cast<unsigned>((a.bs + kTokens - 1) / kTokens)), block(kWaves * kWave);
  const bool through_lds = a.groups > 1 && !lane_groups(a.group_size, kVpl);
  const size_t lds = through_lds ? sizeof(double) * kTokens * (a.num_experts + a.num_experts / kVpl) : 0;
  hipLaunchKernelGGL((route_kernel<kSigmoid, kL, kVpl>), grid, block, lds, stream, a, type);
  return hipGetLastError();
}

template <bool kSigmoid>
hipError_t launch_score(const RouterArgs& a, Out type, hipStream_t stream) {
  return with_router_shape(select::router_shape(a.bs, a.num_experts, a.k), [&](auto lanes, auto vpl) {
    return launch_shape<kSigmoid, decltype(lanes)::value, decltype(vpl)::value>(a, type, stream);
  });
}

}  // namespace

hipError_t launch_route(const RouterArgs& a, Out logits_type, bool sigmoid, hipStream_t stream) {
  for (int64_t first = 0; first < a.bs; first += select::router_launch_tokens()) {
    const RouterArgs part = router_part(a, logits_type, static_cast<int32_t>(first));
    const hipError_t e =
        sigmoid ? launch_score<true>(part, logits_type, stream) : launch_score<false>(part, logits_type, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
