// Expert products in 8-bit floats: e4m3 rows times each expert's e4m3 weights,
// scaled for each 128 of a row (ts) and each 128 x 128 of the weights (ws).
// For a row m of expert g and a column j
//   y[m][j] = sum over the blocks b of k of (ts[m][b] ws[g][j / 128][b]) p_b,
//   p_b = sum over i in block b of a[m][i] w[g][j][i]
// A block's products are summed from zero by the bf16 matrix instructions (the
// codes widened in registers) and added to the binary32 accumulator times the
// block's scale by one multiply-add.  The 8-bit instructions (16x16x128 f8f6f4
// and 16x16x32 fp8) are not as exact: in each eight consecutive products they
// cut what lies below 2^-13 of the largest (measured: 2^3 is kept beside 2^16,
// 2^2 is not), an error of 1.4e-5 of normal rows' results.
//
// The plain form rounds y; the gated form takes 2n columns, gate and up, and
// quantises u g / (1 + e^-g) in blocks of 128 columns (block_rows.h).  A block
// is the work of one workgroup, so nothing but the 8-bit rows leaves the chip.
//
// The weights are the first operand and the rows the second: a lane then holds
// four consecutive columns of one row, and one scale serves all four.
//
// stream_f8_kernel: a workgroup takes kMI x 16 rows; the rows lie in LDS in
// chunks of kKC bytes of k, two buffers; a wave owns 16 columns (16 gate and 16
// up) and loads their weights straight into registers, two chunks ahead, each
// byte once.
#include "block_rows.h"
#include "device_util.h"
#include "gemm.h"
#include "gemm_f8.h"
#include "router_util.h"
#include "row_range.h"
#include "row_slots.h"

#pragma clang fp contract(off)

namespace moe {
namespace {

// u g / (1 + e^-g); e^-g overflows to infinity only where the quotient is 0.
__device__ __forceinline__ float gated(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// Four consecutive columns of one row, as far as the row goes.
template <Form kForm>
__device__ __forceinline__ void store_columns(const GemmF8Args& a, int64_t row, int col, const f32x4& v) {
  constexpr Out kOut = static_cast<Out>(kForm);
  const int64_t at = row * a.n + col;
  if (col + 4 <= a.n) {
    if constexpr (kOut == Out::kF32)
      *reinterpret_cast<f32x4_u*>(static_cast<float*>(a.out) + at) = v;
    else
      *reinterpret_cast<u32x2_u*>(static_cast<uint16_t*>(a.out) + at) =
          u32x2{pack2<kOut == Out::kFp16>(v[0], v[1]), pack2<kOut == Out::kFp16>(v[2], v[3])};
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (col + q < a.n) store_float<kOut>(a.out, at + q, round_f32(v[q]));
  }
}

// ---- few rows for each expert -----------------------------------------------------

template <Form kForm, int kMI, int kWaves, int kKC>
__global__ __launch_bounds__(kWave* kWaves) void stream_f8_kernel(GemmF8Args a, int64_t slots) {
  constexpr bool kGated = kForm == Form::kGated;
  constexpr int kNI = kGated ? 2 : 1;  // fragments of 16 columns of a wave: gate and up
  constexpr int kThreads = kWave * kWaves, kCols = 16 * kWaves, kRows = 16 * kMI;
  constexpr int kRowPieces = kKC / 16, kSteps = kKC / kF8Block;
  constexpr int kCopies = kRows * kRowPieces / kThreads;  // pieces of a chunk's rows that a thread brings
  constexpr int kScales = kRows * kSteps;                 // of a chunk, for each of kNI
  static_assert(kRowPieces % 16 == 0 && kCopies * kThreads == kRows * kRowPieces, "whole chunks");
  static_assert(kScales <= kThreads && kF8Block % kCols == 0, "a scale a thread, one block of columns a workgroup");
  __shared__ __attribute__((aligned(1024))) uint8_t rows[2][kRows * kKC];
  __shared__ float scales[2][kNI][kScales];
  __shared__ float row_max[kGated ? kWaves : 1][kRows];
  const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);
  // workgroups of one block of columns lie on one XCD, an expert's slots next to each other
  const int64_t x = blockIdx.x % 8, y = blockIdx.x / 8;
  const int64_t slot = y % slots, block = y / slots * 8 + x;
  if (block * kCols >= a.n) return;
  RowSlot rs;
  if (!find_row_slot<kRows>(a.group_count, a.groups, a.rows, slot, lane, &rs)) return;

  const int col0 = static_cast<int>(block) * kCols + wave * 16;
  const int piece = lane / 16 * 16, l16 = lane % 16;
  const int kb = f8_blocks(a.k), nb = f8_blocks(a.n);
  const uint8_t* pb[kNI];
  const float* ws[kNI];
#pragma unroll
  for (int j = 0; j < kNI; ++j) {
    const int64_t half = static_cast<int64_t>(rs.group) * kNI + j;
    pb[j] = a.w + (half * a.n + min(col0 + l16, a.n - 1)) * a.k;
    ws[j] = a.weight_scale + (half * nb + static_cast<int>(block) * kCols / kF8Block) * kb;
  }
  const uint8_t* pa[kCopies];
  int ka[kCopies], la[kCopies];
#pragma unroll
  for (int q = 0; q < kCopies; ++q) {
    const int p = q * kThreads + tid, r = p / kRowPieces, c = p % kRowPieces;
    pa[q] = a.a + tile_row(rs.row0, rs.row_end, r) * a.a_stride;
    ka[q] = c * 16;
    la[q] = r * kKC + (c ^ (r % 16)) * 16;
  }
  // scale tid of a chunk: step tid / kRows, row tid % kRows
  const int sr = tid % kRows, sb = tid / kRows;
  const float* pts = reinterpret_cast<const float*>(
      a.token_scale + static_cast<int64_t>(tile_row(rs.row0, rs.row_end, sr)) * a.ts_stride);
  const int rounds = (a.k + kKC - 1) / kKC;
  // Past k the rows' codes count as zero, and so do their scales; the weights there are some of the same column's.
  struct Codes {
    i32x4 a, b;
  };
  struct Rows {
    i32x4 v[kCopies];
    float s[kNI];
  };
  auto load_a = [&](int chunk, Rows& to) {
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const int at = chunk * kKC + ka[q];
      to.v[q] = *reinterpret_cast<const i32x4*>(pa[q] + (at < a.k ? at : 0));
      if (at >= a.k) to.v[q] = i32x4{0, 0, 0, 0};
    }
    const int b = chunk * kSteps + sb;
    const bool have = tid < kScales && b < kb;
    const float ts = have ? pts[b] : 0.0f;
#pragma unroll
    for (int j = 0; j < kNI; ++j) to.s[j] = have ? ts * ws[j][b] : 0.0f;
  };
  auto put_a = [&](int buf, const Rows& from) {
#pragma unroll
    for (int q = 0; q < kCopies; ++q) *reinterpret_cast<i32x4*>(rows[buf] + la[q]) = from.v[q];
#pragma unroll
    for (int j = 0; j < kNI; ++j)
      if (tid < kScales) scales[buf][j][tid] = from.s[j];
  };
  auto load_b = [&](int chunk, Codes (&v)[kSteps][kNI]) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int at = chunk * kKC + s * kF8Block + piece;
#pragma unroll
      for (int j = 0; j < kNI; ++j)
        v[s][j] = Codes{*reinterpret_cast<const i32x4*>(pb[j] + (at < a.k ? at : 0)),
                        *reinterpret_cast<const i32x4*>(pb[j] + (at + 64 < a.k ? at + 64 : 0))};
    }
  };
  f32x4 acc[kMI][kNI];
#pragma unroll
  for (int i = 0; i < kMI; ++i)
#pragma unroll
    for (int j = 0; j < kNI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](int buf, const Codes (&b)[kSteps][kNI]) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      WideCodes w[kNI];
#pragma unroll
      for (int j = 0; j < kNI; ++j) w[j] = widen(b[s][j].a, b[s][j].b);
#pragma unroll
      for (int i = 0; i < kMI; ++i) {
        const uint8_t* row = rows[buf] + (i * 16 + l16) * kKC;
        const WideCodes f = widen(*reinterpret_cast<const i32x4*>(row + ((s * 8 + lane / 16) ^ l16) * 16),
                                  *reinterpret_cast<const i32x4*>(row + ((s * 8 + 4 + lane / 16) ^ l16) * 16));
#pragma unroll
        for (int j = 0; j < kNI; ++j) {
          const f32x4 p = block_sum(w[j], f);
          const float scale = scales[buf][j][s * kRows + i * 16 + l16];
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(p[q], scale, acc[i][j][q]);
        }
      }
    }
  };

  Rows a0, a1;
  Codes b0[kSteps][kNI], b1[kSteps][kNI];
  load_a(0, a0);
  load_b(0, b0);
  if (rounds > 1) {
    load_a(1, a1);
    load_b(1, b1);
  }
  put_a(0, a0);
  __syncthreads();
  // A buffer is written again only after the barrier that follows its readers.
  for (int c = 0;; c += 2) {
    multiply(0, b0);
    if (c + 1 >= rounds) break;
    if (c + 2 < rounds) {
      load_a(c + 2, a0);
      load_b(c + 2, b0);
    }
    put_a(1, a1);
    __syncthreads();
    multiply(1, b1);
    if (c + 2 >= rounds) break;
    if (c + 3 < rounds) {
      load_a(c + 3, a1);
      load_b(c + 3, b1);
    }
    put_a(0, a0);
    __syncthreads();
  }

  const int col = col0 + lane / 16 * 4;
  if constexpr (!kGated) {
    if (col >= a.n) return;
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
      const int r = i * 16 + l16;
      if (tile_has_row(rs.row0, rs.row_end, r)) store_columns<kForm>(a, rs.row0 + r, col, acc[i][0]);
    }
  } else {
    // n is a multiple of 16: a wave's columns all exist, or none does
    float act[kMI][4];
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
      float m = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        act[i][q] = gated(acc[i][0][q], acc[i][1][q]);
        m = __builtin_fmaxf(m, __builtin_fabsf(act[i][q]));
      }
      m = __builtin_fmaxf(m, __shfl_xor(m, 16));
      m = __builtin_fmaxf(m, __shfl_xor(m, 32));
      if (lane < 16) row_max[wave][i * 16 + lane] = col0 < a.n ? m : 0.0f;
    }
    __syncthreads();
    if (col0 >= a.n) return;
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
      const int r = i * 16 + l16;
      float m = 0.0f;
#pragma unroll
      for (int v = 0; v < kWaves; ++v) m = __builtin_fmaxf(m, row_max[v][r]);
      float scale, factor;
      f8_scale(m, scale, factor);
      if (!tile_has_row(rs.row0, rs.row_end, r)) continue;
      uint8_t* dst = static_cast<uint8_t*>(a.out) + static_cast<int64_t>(rs.row0 + r) * a.out_row_bytes;
      *reinterpret_cast<uint32_t*>(dst + col) =
          f8_pack4(act[i][0] * factor, act[i][1] * factor, act[i][2] * factor, act[i][3] * factor);
      if (wave == 0 && lane < 16) *reinterpret_cast<float*>(dst + a.out_scale_off + block * 4) = scale;
    }
  }
}

int64_t stream_blocks(int32_t rows, int32_t groups, int32_t n, int tile_m, int tile_n) {
  return row_slots(rows, groups, tile_m) * (((static_cast<int64_t>(n) + tile_n - 1) / tile_n + 7) / 8 * 8);
}

template <Form kForm, int kMI, int kWaves, int kKC>
hipError_t launch_stream(const GemmF8Args& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(stream_blocks(a.rows, a.groups, a.n, kMI * 16, 16 * kWaves)));
  stream_f8_kernel<kForm, kMI, kWaves, kKC>
      <<<grid, dim3(kWave * kWaves), 0, stream>>>(a, row_slots(a.rows, a.groups, kMI * 16));
  return hipGetLastError();
}

}  // namespace

bool grouped_gemm_f8_fits(int32_t rows, int32_t groups, int32_t n, bool swiglu) {
  const int64_t blocks = stream_blocks(rows, groups, n, 32, swiglu ? 128 : 64);
  return blocks <= kMaxLaunchThreads / (kWave * (swiglu ? 8 : 4));
}

hipError_t launch_grouped_gemm_f8(const GemmF8Args& a, Out out_type, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  switch (out_type) {
    case Out::kBf16: return launch_stream<Form::kBf16, 2, 4, 256>(a, stream);
    case Out::kFp16: return launch_stream<Form::kFp16, 2, 4, 256>(a, stream);
    case Out::kF32: return launch_stream<Form::kF32, 2, 4, 256>(a, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_grouped_gemm_swiglu_quant_f8(const GemmF8Args& a, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  return launch_stream<Form::kGated, 2, 8, 256>(a, stream);
}

}  // namespace moe
