// Second expert matmul of the MoE layer's expert side (GMM2): int8 rows times
// each expert's int8 weights, scaled by token and by output channel
// ("UMDK/CAM communication acceleration library deep analysis v2", section
// 4.3).  For a row m of expert g and a column j
//   out[m][j] = round((float(sum_i a[m][i] w[g][j][i]) * ws[g][j]) * ts_m)
// with the sum exact in int32 (below 2^31 for any order) and each later
// operation rounded to binary32, so the result does not depend on the tiling.
//
// One wave per 16 x 16 tile of one expert's output, straight from global
// memory: in a step of 64 k bytes lane l holds 16 bytes of row (column) l % 16
// at k offset 16 (l / 16) for v_mfma_i32_16x16x64_i8.
#include "device_util.h"
#include "gemm.h"
#include "router_util.h"
#include "row_slots.h"

#pragma clang fp contract(off)

namespace moe {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 16, kStepK = 64, kWaves = 4;

template <Out kOut>
__global__ __launch_bounds__(kWave* kWaves) void grouped_gemm_deq_kernel(GemmDeqArgs a) {
  const int lane = threadIdx.x % kWave, wave = uniform(static_cast<int>(threadIdx.x / kWave));
  const int64_t col_blocks = (a.n + kTile * kWaves - 1) / (kTile * kWaves);
  const int64_t slot = blockIdx.x / col_blocks;
  const int col0 = static_cast<int>(blockIdx.x - slot * col_blocks) * kTile * kWaves + wave * kTile;
  RowSlot rs;
  if (!find_row_slot<kTile>(a.group_count, a.groups, a.rows, slot, lane, &rs) || col0 >= a.n) return;

  const int piece = lane / 16 * 16;
  const int8_t* pa = a.a + min(rs.row0 + lane % 16, rs.row_end - 1) * a.a_stride;
  const int col = col0 + lane % 16;
  const int8_t* pb = a.w + (static_cast<int64_t>(rs.group) * a.n + min(col, a.n - 1)) * a.k;
  i32x4 acc = {0, 0, 0, 0};
  for (int k0 = 0; k0 < a.k; k0 += kStepK) {
    const bool in = k0 + piece < a.k;  // k ends inside the step: the rest of the row of a counts as zero
    const int at = in ? k0 + piece : 0;
    i32x4 fa = *reinterpret_cast<const i32x4*>(pa + at);
    const i32x4 fb = *reinterpret_cast<const i32x4*>(pb + at);
    if (!in) fa = i32x4{0, 0, 0, 0};
    acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa, fb, acc, 0, 0, 0);
  }
  if (col >= a.n) return;
  const float ws = a.weight_scale[static_cast<int64_t>(rs.group) * a.n + col];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = rs.row0 + lane / 16 * 4 + r;
    if (row < rs.row_end) {
      const float ts = *reinterpret_cast<const float*>(a.token_scale + row * a.ts_stride);
      store_float<kOut>(a.out, static_cast<int64_t>(row) * a.n + col, round_f32(static_cast<float>(acc[r]) * ws * ts));
    }
  }
}

}  // namespace

int64_t grouped_gemm_deq_blocks(int32_t rows, int32_t groups, int32_t n, int32_t k) {
  (void)k;
  return row_slots(rows, groups, kTile) * ((static_cast<int64_t>(n) + kTile * kWaves - 1) / (kTile * kWaves));
}

hipError_t launch_grouped_gemm_deq(const GemmDeqArgs& a, Out out_type, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  const int64_t blocks = grouped_gemm_deq_blocks(a.rows, a.groups, a.n, a.k);
  if (blocks > kGemmMaxBlocks) return hipErrorInvalidValue;
  const dim3 grid(static_cast<uint32_t>(blocks)), block(kWave * kWaves);
  switch (out_type) {
    case Out::kBf16: grouped_gemm_deq_kernel<Out::kBf16><<<grid, block, 0, stream>>>(a); break;
    case Out::kFp16: grouped_gemm_deq_kernel<Out::kFp16><<<grid, block, 0, stream>>>(a); break;
    case Out::kF32: grouped_gemm_deq_kernel<Out::kF32><<<grid, block, 0, stream>>>(a); break;
  }
  return hipGetLastError();
}

}  // namespace moe
