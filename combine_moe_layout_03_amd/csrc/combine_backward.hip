// The gradient of the combine: for the entries (t, j) of token t, with g its
// output gradient and y the entry's receive row,
//   row gradient = round(w_tj * g),   weight gradient = sum_i y[i] * g[i].
//
// A wave an entry, up to eight entries of a token in a workgroup (which share g
// through the caches), or 16 lanes an entry where the rows are short
// (select_layer.h).  A lane owns chunks of 8 elements, a wave's lanes a
// contiguous 1 KB; it reads y and g, adds to its sum and stores the row
// gradient in y's place, so a row may be replaced in place.  A sum is a
// lane's even and odd chunks in order, both, then the lanes: a fixed order.
//
// Bound by the rows' bytes: 4096 tokens x 8 entries, h 7168, bf16, 195 us for
// 0.999 GB = 5.1 TB/s (a large copy_ of torch 5.1-5.3, its elementwise kernel
// with one read and one write stream 6.2).  (A workgroup per token that takes its
// rows together: 211 us; row by row with g in registers: 193-204.)  The rows are
// loaded non-temporally, and stored so where they are more than the Infinity
// Cache keeps (select_layer.h); that instance has a wave an entry whatever the
// rows' length.
#include "device_util.h"
#include "layer.h"
#include "router_util.h"

#pragma clang fp contract(off)

namespace moe {
namespace {

constexpr int kMaxWaves = 8;  // of a workgroup
constexpr int kUnroll = 2;    // chunks in flight per lane, with a sum each

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

// Byte offset of an entry's receive row, -1 where it has none.
__device__ __forceinline__ int64_t entry_row(const RouteArgs& a, int entry) {
  const int e = a.topk_idx[entry], slot = a.send_token_idx[entry];
  const int ec = min(max(e, 0), a.num_experts - 1);
  const int rank = static_cast<int>((static_cast<uint64_t>(ec) * a.epr_magic) >> 32);
  const int64_t row = static_cast<int64_t>(a.recv_base[rank]) + a.put_offset[ec * a.put_stride] + slot;
  const bool ok = ec == e && slot >= 0 && row >= 0 && row < a.cap_rows;
  return ok ? row * a.row_bytes : -1;
}

template <int kL, bool kFp16, Out kGrad, bool kNtStore>
__global__ __launch_bounds__(kWave* kMaxWaves) void combine_backward_kernel(RouteArgs a, const void* grad_out,
                                                                         const uint8_t* recv, const float* topk_w,
                                                                         uint8_t* grad_recv, float* grad_w) {
  const int lane = threadIdx.x % kL;
  const uint32_t count = static_cast<uint32_t>(a.bs) * static_cast<uint32_t>(a.k);  // below 2^31
  uint32_t mine = blockIdx.x * (blockDim.x / kL) + threadIdx.x / kL;
  if constexpr (kL == kWave) mine = static_cast<uint32_t>(uniform(static_cast<int>(mine)));
  const bool active = mine < count;
  const int entry = static_cast<int>(min(mine, count - 1));  // lanes past the last entry store nothing
  const int t = static_cast<int>(static_cast<uint32_t>(entry) / static_cast<uint32_t>(a.k));
  const int64_t off = entry_row(a, entry);
  const float w = topk_w[entry];
  const int chunks = a.hidden >> 3;
  float sums[kUnroll] = {};
  if (active && off >= 0) {
    for (int c0 = lane; c0 < chunks; c0 += kL * kUnroll) {
      u32x4 y[kUnroll];
      float g[kUnroll][8];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {  // (past the row's end its last chunk, which is not used)
        const int c = min(c0 + u * kL, chunks - 1);
        y[u] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(recv + off + c * 16));
        load_grad<kGrad>(grad_out, static_cast<int64_t>(t) * a.hidden + c * 8, g[u]);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int c = c0 + u * kL;
        if (c >= chunks) break;
        float f[8];
        widen<kFp16>(y[u], f);
#pragma unroll
        for (int q = 0; q < 8; ++q) sums[u] = __builtin_fmaf(f[q], g[u][q], sums[u]);
        u32x4 d;
#pragma unroll
        for (int q = 0; q < 4; ++q) d[q] = pack2<kFp16>(w * g[u][2 * q], w * g[u][2 * q + 1]);
        u32x4* dst = reinterpret_cast<u32x4*>(grad_recv + off + c * 16);
        if constexpr (kNtStore) __builtin_nontemporal_store(d, dst);
        else *dst = d;
      }
    }
  }
  const float sum = token_sum<kL>(sums[0] + sums[1]);
  if (active && lane == 0) grad_w[entry] = sum;
}

template <int kL, bool kFp16, Out kGrad, bool kNtStore>
hipError_t launch_shape(const RouteArgs& r, const void* grad_out, const uint8_t* recv, const float* topk_w,
                        uint8_t* grad_recv, float* grad_w, hipStream_t stream) {
  // a workgroup for a token's entries, or for an even part of them (9 entries, h
  // 2208, 428 tokens: 12.1 us, and 14.5 as 8 and 1)
  const int parts = (r.k + kMaxWaves - 1) / kMaxWaves, waves = kL == kWave ? (r.k + parts - 1) / parts : kMaxWaves;
  const int64_t entries = static_cast<int64_t>(kWave / kL) * waves;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(r.bs) * r.k + entries - 1) / entries));
  hipLaunchKernelGGL((combine_backward_kernel<kL, kFp16, kGrad, kNtStore>), grid, dim3(kWave * waves), 0, stream, r,
                     grad_out, recv, topk_w, grad_recv, grad_w);
  return hipGetLastError();
}

template <bool kFp16, Out kGrad>
hipError_t launch_grad(const RouteArgs& r, const void* grad_out, const uint8_t* recv, const float* topk_w,
                       uint8_t* grad_recv, float* grad_w, hipStream_t stream) {
  if (select::combine_backward_nt(int64_t(r.bs) * r.k * r.row_bytes))
    return launch_shape<64, kFp16, kGrad, true>(r, grad_out, recv, topk_w, grad_recv, grad_w, stream);
  if (select::combine_backward_short(r.hidden))
    return launch_shape<16, kFp16, kGrad, false>(r, grad_out, recv, topk_w, grad_recv, grad_w, stream);
  return launch_shape<64, kFp16, kGrad, false>(r, grad_out, recv, topk_w, grad_recv, grad_w, stream);
}

template <bool kFp16>
hipError_t launch_rows(const RouteArgs& r, const void* grad_out, Out grad_type, const uint8_t* recv,
                       const float* topk_w, uint8_t* grad_recv, float* grad_w, hipStream_t stream) {
  switch (grad_type) {
    case Out::kBf16: return launch_grad<kFp16, Out::kBf16>(r, grad_out, recv, topk_w, grad_recv, grad_w, stream);
    case Out::kFp16: return launch_grad<kFp16, Out::kFp16>(r, grad_out, recv, topk_w, grad_recv, grad_w, stream);
    case Out::kF32: return launch_grad<kFp16, Out::kF32>(r, grad_out, recv, topk_w, grad_recv, grad_w, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_combine_backward(const RouteArgs& r, const void* grad_out, Out grad_type, const void* recv_x,
                                   Half recv_type, const float* topk_w, void* grad_recv, float* grad_weights,
                                   hipStream_t stream) {
  const uint8_t* recv = static_cast<const uint8_t*>(recv_x);
  uint8_t* grad = static_cast<uint8_t*>(grad_recv);
  const int64_t grad_row = static_cast<int64_t>(r.hidden) * (grad_type == Out::kF32 ? 4 : 2);
  const int32_t tokens = select::combine_backward_launch_tokens(r.k);
  for (int64_t first = 0; first < r.bs; first += tokens) {
    RouteArgs part = r;
    part.bs = static_cast<int32_t>(r.bs - first < tokens ? r.bs - first : tokens);
    part.topk_idx += first * r.k;
    part.send_token_idx += first * r.k;
    const void* g = static_cast<const uint8_t*>(grad_out) + first * grad_row;
    const float* w = topk_w + first * r.k;
    float* gw = grad_weights + first * r.k;
    const hipError_t e = recv_type == Half::kFp16
                             ? launch_rows<true>(part, g, grad_type, recv, w, grad, gw, stream)
                             : launch_rows<false>(part, g, grad_type, recv, w, grad, gw, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
