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
#include "select_f8.h"
#include "select_layer.h"

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

// ---- many rows for each expert -----------------------------------------------------

constexpr int kTileWaves = 8;
constexpr int kSK = kF8Block;     // bytes of k per stage: one block
constexpr int kRound = 6;         // stages of a round: the slots' places come round again
constexpr int kGroupCols = 1024;  // rows of weights of a group of column tiles

constexpr int vmcnt_wait(int n) { return 0x0f70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kLgkmWait0 = 0xc07f;
#define MOE_LDS __attribute__((address_space(3)))

// Position of a 16-byte piece in a stage row: piece p of row r sits at p ^
// swizzle(r).  The fragments read 16 rows at one piece, rows 16 i + (0 .. 15)
// of the rows and 32 p + {0-3, 8-11, 16-19, 24-27} (+ 4) of the weights; for
// both the 16 rows fall into all 16 groups of banks.
__device__ __forceinline__ int swizzle(int r) { return ((r >> 1) & 7) ^ (((r >> 4) & 1) << 1); }

// Lane l's value is that of row l of a wave's 64 rows (of l % 32 with 32): in
// every lane, for each fragment i, the value of row 16 i + l % 16.
template <int kMI>
__device__ __forceinline__ void spread_rows(float v, float (&to)[kMI]) {
  static_assert(kMI == 2 || kMI == 4, "32 or 64 rows");
  const uint32_t b = __float_as_uint(v);
  const auto h = __builtin_amdgcn_permlane16_swap(b, b, false, false);  // rows 0 0 2 2 and 1 1 3 3
  if constexpr (kMI == 2) {
    to[0] = __uint_as_float(h[0]), to[1] = __uint_as_float(h[1]);
  } else {
    const auto even = __builtin_amdgcn_permlane32_swap(h[0], h[0], false, false);
    const auto odd = __builtin_amdgcn_permlane32_swap(h[1], h[1], false, false);
    to[0] = __uint_as_float(even[0]), to[1] = __uint_as_float(odd[0]);
    to[2] = __uint_as_float(even[1]), to[3] = __uint_as_float(odd[1]);
  }
}

// 16 bytes of consecutive columns of one row, as far as the row goes.
template <Form kForm>
__device__ __forceinline__ void store_piece(const GemmF8Args& a, int64_t row, int col, const u32x4& bits) {
  constexpr int kSize = kForm == Form::kF32 ? 4 : 2, kCols = 16 / kSize;
  const int64_t at = row * a.n + col;
  if (col + kCols <= a.n) {
    u32x4_u* const dst = reinterpret_cast<u32x4_u*>(static_cast<uint8_t*>(a.out) + at * kSize);
    if (a.nt) {  // the marks keep the compiler from joining the two into one ordinary store
      asm volatile("; non-temporal");
      __builtin_nontemporal_store(bits, dst);
      asm volatile("; non-temporal");
    } else {
      *dst = bits;
    }
  } else {
#pragma unroll
    for (int q = 0; q < kCols; ++q) {
      if (col + q >= a.n) continue;
      if constexpr (kForm == Form::kF32) static_cast<uint32_t*>(a.out)[at + q] = bits[q];
      else static_cast<uint16_t*>(a.out)[at + q] = static_cast<uint16_t>(bits[q / 2] >> (q % 2 * 16));
    }
  }
}

template <bool kWide>
struct Fragment;
template <>
struct Fragment<true> {
  WideCodes c;
  __device__ __forceinline__ void set(i32x4 a, i32x4 b) { c = widen(a, b); }
};
template <>
struct Fragment<false> {
  i32x8 c;
  __device__ __forceinline__ void set(i32x4 a, i32x4 b) { c = join(a, b); }
};
// The block's sums of one fragment of weights with kMI of rows, the chains of
// instructions side by side.
template <int kMI>
__device__ __forceinline__ void block_sums(const Fragment<true>& w, const Fragment<true> (&a)[kMI], f32x4 (&p)[kMI]) {
#pragma unroll
  for (int i = 0; i < kMI; ++i) p[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < kMI; ++i) p[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.c.v[q], a[i].c.v[q], p[i], 0, 0, 0);
}
template <int kMI>
__device__ __forceinline__ void block_sums(const Fragment<false>& w, const Fragment<false> (&a)[kMI], f32x4 (&p)[kMI]) {
#pragma unroll
  for (int i = 0; i < kMI; ++i) p[i] = block_sum(w.c, a[i].c);
}

template <Form kForm, bool kWide, int kTileM, int kTileN, int kWavesM, bool kTail>
__global__ __launch_bounds__(kWave* kTileWaves) void tile_f8_kernel(GemmF8Args a) {
  constexpr bool kGated = kForm == Form::kGated;
  constexpr int kHalves = kGated ? 2 : 1;  // gate and up
  constexpr int kWavesN = kTileWaves / kWavesM;
  constexpr int kWaveM = kTileM / kWavesM, kWaveN = kTileN / kWavesN;
  constexpr int kMI = kWaveM / 16, kNI = kWaveN / 16, kStepNI = kNI / 2;
  constexpr int kCols = kTileN / kHalves;  // columns of the result
  constexpr int kRowsPerLoad = kWave / (kSK / 16);
  constexpr int kLoadsA = kTileM / kRowsPerLoad / kTileWaves, kLoadsB = kTileN / kRowsPerLoad / kTileWaves;
  static_assert(kF8Block % (kWaveN / kHalves) == 0 && (!kGated || kCols == kF8Block), "a wave's columns share a scale");
  __shared__ __attribute__((aligned(1024))) uint8_t sa0[kTileM * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sa1[kTileM * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sb0[kTileN * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sb1[kTileN * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sb2[kTileN * kSK];
  const int tid = threadIdx.x, lane = tid % kWave, wave = uniform(tid / kWave);

  // Tiles in order: groups of column tiles, the row slots of a group, its
  // columns; XCD x (workgroups x, x + 8, ...) takes the x-th eighth of the
  // tiles that the counts give.
  constexpr int kGroup = kGroupCols / kTileN;
  const int64_t n_tiles = (a.n + kCols - 1) / kCols;
  int64_t col_tile = 0;
  const auto pick = [&](int64_t slots) -> int64_t {
    const int64_t tiles = n_tiles * slots, per_xcd = (tiles + 7) / 8;
    const int64_t l = blockIdx.x / 8, t = blockIdx.x % 8 * per_xcd + l;
    if (l >= per_xcd || t >= tiles) return -1;
    const int64_t group = t / (slots * kGroup), within = t - group * slots * kGroup;
    const int64_t width = min(n_tiles - group * kGroup, static_cast<int64_t>(kGroup));
    col_tile = group * kGroup + within % width;
    return within / width;
  };
  RowSlot rs;
  if (!place_row_slot<kTileM>(a.group_count, a.groups, a.rows, lane, pick, &rs)) return;  // the whole workgroup
  const int row0 = rs.row0, row_end = rs.row_end;
  const int col0 = static_cast<int>(col_tile) * kCols;
  const int wm = wave / kWavesN, wn = wave % kWavesN;
  const int l16 = lane % 16;

  // Load q of this wave fills the stage rows from 8 (q 8 + wave); lane l
  // fetches the piece that belongs at position l % 8 of row l / 8, the same
  // piece for every q.  A wave's stage rows of weights are its gate rows, then
  // its up rows.
  const int piece = (lane % 8) ^ swizzle(kRowsPerLoad * wave + lane / 8);
  // Offsets from the tile's first row fit in 32 bits: 256 rows of at most
  // kF8MaxRowBytes, and weights of at most 2^16 columns by 2^16 with 256 more.
  const uint8_t* const base_a = a.a + row0 * a.a_stride;
  const uint8_t* const base_b = a.w + (static_cast<int64_t>(rs.group) * kHalves * a.n + col0) * a.k;
  uint32_t src_a[kLoadsA], src_b[kLoadsB];
#pragma unroll
  for (int q = 0; q < kLoadsA; ++q) {
    const int r = kRowsPerLoad * (q * kTileWaves + wave) + lane / 8;
    src_a[q] = static_cast<uint32_t>(tile_row(row0, row_end, r) - row0) * static_cast<uint32_t>(a.a_stride) + piece * 16;
  }
#pragma unroll
  for (int q = 0; q < kLoadsB; ++q) {
    const int r = kRowsPerLoad * (q * kTileWaves + wave) + lane / 8;
    constexpr int kPart = kWaveN / kHalves;
    const int half = r % kWaveN / kPart, c = r / kWaveN * kPart + r % kPart;
    src_b[q] = static_cast<uint32_t>(half * a.n + min(c, a.n - 1 - col0)) * static_cast<uint32_t>(a.k) + piece * 16;
  }
  // The scales: lane l has those of the wave's row l, two stages ahead; the
  // weights' are the same in every lane, and come a round's at a time.
  const int stages = f8_blocks(a.k), nb = f8_blocks(a.n);
  const float* const ts_row = reinterpret_cast<const float*>(
      a.token_scale + static_cast<int64_t>(tile_row(row0, row_end, wm * kWaveM + lane % kWaveM)) * a.ts_stride);
  const int col_block = uniform(min((col0 + wn * (kWaveN / kHalves)) / kF8Block, nb - 1));
  const float* ws[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
    ws[h] = a.weight_scale + ((static_cast<int64_t>(rs.group) * kHalves + h) * nb + col_block) * stages;
  float row_scale[2];  // of this stage and the next
  struct ColScales {
    float v[kHalves][kRound];
  };
  const auto load_col_scales = [&](int first, ColScales& s) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
#pragma unroll
      for (int q = 0; q < kRound; ++q) s.v[h][q] = ws[h][min(first + q, stages - 1)];
  };
  // Stages past the last one load it again, into slots that are not read; a
  // piece past k reads the row's first piece (its row fragments count as zero).
  auto stage_offset = [&](int s) {
    return min(s, stages - 1) * kSK;
  };
  auto tail_offset = [&](int k0) { return static_cast<uint32_t>((k0 + piece * 16 < a.k) ? k0 : -piece * 16); };
  auto issue_a = [&](int s, uint8_t* buf) {
    const int k0 = stage_offset(s);
#pragma unroll
    for (int q = 0; q < kLoadsA; ++q) {
      const uint8_t* src;
      if constexpr (kTail) src = base_a + (src_a[q] + tail_offset(k0));
      else src = base_a + k0 + src_a[q];
      __builtin_amdgcn_global_load_lds(src, (MOE_LDS void*)(buf + (q * kTileWaves + wave) * kRowsPerLoad * kSK), 16, 0,
                                       0);
    }
  };
  auto issue_b = [&](int s, uint8_t* buf) {
    const int k0 = stage_offset(s);
#pragma unroll
    for (int q = 0; q < kLoadsB; ++q) {
      const uint8_t* src;
      if constexpr (kTail) src = base_b + (src_b[q] + tail_offset(k0));
      else src = base_b + k0 + src_b[q];
      __builtin_amdgcn_global_load_lds(src, (MOE_LDS void*)(buf + (q * kTileWaves + wave) * kRowsPerLoad * kSK), 16, 0,
                                       0);
    }
  };

  const int frag_a = (wm * kWaveM + l16) * kSK;
  // pair p, tile t of the weights: row 32 p + 8 (l16 / 4) + 4 t + l16 % 4, so
  // that a lane ends with 8 consecutive columns in the two tiles
  const int row_b = 8 * (l16 / 4) + l16 % 4;
  const int frag_b = (wn * kWaveN + row_b) * kSK;
  const int swz_a = swizzle(l16), swz_b = swizzle(row_b);
  f32x4 acc[kMI][kNI];
#pragma unroll
  for (int i = 0; i < kMI; ++i)
#pragma unroll
    for (int j = 0; j < kNI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  auto barrier = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
  };
  Fragment<kWide> af[kMI];
  // Half of a stage's columns: with a gate, its gate or its up columns.
  auto step = [&](int S, int h, float ts, float w, const uint8_t* ca, const uint8_t* cb, uint8_t* fill_a,
                  uint8_t* fill_b) {
    if (h == 0) issue_a(S + 1, fill_a);  // into the slot A(S - 1) used
    else issue_b(S + 2, fill_b);         // into the slot B(S - 1) used
    const int p = lane / 16;
    i32x4 ra[kMI][2], rb[kStepNI][2];
    if (h == 0) {
#pragma unroll
      for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q)
          ra[i][q] = *reinterpret_cast<const i32x4*>(ca + frag_a + i * 16 * kSK +
                                                     ((4 * q + p) ^ swz_a ^ ((i & 1) << 1)) * 16);
    }
#pragma unroll
    for (int n = 0; n < kStepNI; ++n) {
      const int j = h * kStepNI + n;
#pragma unroll
      for (int q = 0; q < 2; ++q)
        rb[n][q] = *reinterpret_cast<const i32x4*>(cb + frag_b + ((j >> 1) * 32 + (j & 1) * 4) * kSK +
                                                   ((4 * q + p) ^ swz_b ^ ((j & 1) << 1)) * 16);
    }
    float s[kMI];
    spread_rows<kMI>(ts, s);
#pragma unroll
    for (int i = 0; i < kMI; ++i) s[i] *= w;
    // this wave's loads of A(S + 1) and B(S + 1); those of B(S + 2) may still run
    if (h == 1) __builtin_amdgcn_s_waitcnt(vmcnt_wait(kLoadsB));
    __builtin_amdgcn_s_waitcnt(kLgkmWait0);
    if (h == 0) {
#pragma unroll
      for (int i = 0; i < kMI; ++i) {
        if constexpr (kTail) {
#pragma unroll
          for (int q = 0; q < 2; ++q) ra[i][q] &= S * kSK + (4 * q + p) * 16 < a.k ? -1 : 0;
        }
        af[i].set(ra[i][0], ra[i][1]);
      }
    }
    Fragment<kWide> bf[kStepNI];
#pragma unroll
    for (int n = 0; n < kStepNI; ++n) bf[n].set(rb[n][0], rb[n][1]);
    barrier();
#pragma unroll
    for (int n = 0; n < kStepNI; ++n) {
      f32x4 part[kMI];
      block_sums<kMI>(bf[n], af, part);
#pragma unroll
      for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[i][h * kStepNI + n][q] = __builtin_fmaf(part[i][q], s[i], acc[i][h * kStepNI + n][q]);
    }
    barrier();
  };
  auto stage = [&](int S, int u, const ColScales& s, const uint8_t* ca, const uint8_t* cb, uint8_t* fill_a,
                   uint8_t* fill_b) {
    step(S, 0, row_scale[u % 2], s.v[0][u], ca, cb, fill_a, fill_b);
    step(S, 1, row_scale[u % 2], s.v[kHalves - 1][u], ca, cb, fill_a, fill_b);
    row_scale[u % 2] = ts_row[min(S + 2, stages - 1)];
  };
  ColScales now, next;
  load_col_scales(0, next);
#pragma unroll
  for (int u = 0; u < 2; ++u) row_scale[u] = ts_row[min(u, stages - 1)];
  issue_b(0, sb0);
  issue_a(0, sa0);
  issue_b(1, sb1);
  __builtin_amdgcn_s_waitcnt(vmcnt_wait(kLoadsB));
  barrier();
  const int grp = wave / 4;
  if (grp == 1) barrier();  // the second group runs half a step behind
  const int rounds = stages / kRound;
  for (int r = 0; r < rounds; ++r) {
    now = next;
    load_col_scales(kRound * (r + 1), next);
    stage(kRound * r, 0, now, sa0, sb0, sa1, sb2);
    stage(kRound * r + 1, 1, now, sa1, sb1, sa0, sb0);
    stage(kRound * r + 2, 2, now, sa0, sb2, sa1, sb1);
    stage(kRound * r + 3, 3, now, sa1, sb0, sa0, sb2);
    stage(kRound * r + 4, 4, now, sa0, sb1, sa1, sb0);
    stage(kRound * r + 5, 5, now, sa1, sb2, sa0, sb1);
  }
  {
    const int rest = stages - rounds * kRound;
    if (rest > 0) stage(kRound * rounds, 0, next, sa0, sb0, sa1, sb2);
    if (rest > 1) stage(kRound * rounds + 1, 1, next, sa1, sb1, sa0, sb0);
    if (rest > 2) stage(kRound * rounds + 2, 2, next, sa0, sb2, sa1, sb1);
    if (rest > 3) stage(kRound * rounds + 3, 3, next, sa1, sb0, sa0, sb2);
    if (rest > 4) stage(kRound * rounds + 4, 4, next, sa0, sb1, sa1, sb0);
  }
  if (grp == 0) barrier();  // every wave passes the same number of barriers
  // no load may still be writing this workgroup's LDS
  __builtin_amdgcn_s_waitcnt(vmcnt_wait(0));
  // The results pass through LDS, so that a store's lanes lie along rows (whole
  // cache lines).  The slots are free once every wave's loads have landed and
  // its reads are done.
  barrier();
  if constexpr (!kGated) {
    constexpr int kPieceCols = kForm == Form::kF32 ? 4 : 8;  // columns of a 16-byte piece
    constexpr int kRowPieces = kWaveN / kPieceCols, kWaveBytes = 16 * kRowPieces * 16;
    constexpr int kSlotWaves = kTileN * kSK / kWaveBytes < kTileWaves ? kTileN * kSK / kWaveBytes : kTileWaves;
    static_assert(2 * kSlotWaves >= kTileWaves, "two slots hold every wave's rows");
    uint8_t* const mine = (wave < kSlotWaves ? sb0 : sb1) + wave % kSlotWaves * kWaveBytes;
    // piece c of row r lies at c ^ r, so that 16 rows' pieces fall into all banks
    constexpr int kTurn = (kRowPieces < 16 ? kRowPieces : 16) - 1;
    const auto place = [&](int r, int c) { return mine + (r * kRowPieces + (c ^ (r & kTurn))) * 16; };
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
#pragma unroll
      for (int p = 0; p < kNI / 2; ++p) {
        const f32x4 v = acc[i][2 * p], u = acc[i][2 * p + 1];
        const int c = (p * 4 + lane / 16) * (8 / kPieceCols);
        if constexpr (kForm == Form::kF32) {
          *reinterpret_cast<f32x4*>(place(l16, c)) = v;
          *reinterpret_cast<f32x4*>(place(l16, c + 1)) = u;
        } else {
          constexpr bool kFp16 = kForm == Form::kFp16;
          *reinterpret_cast<u32x4*>(place(l16, c)) = u32x4{pack2<kFp16>(v[0], v[1]), pack2<kFp16>(v[2], v[3]),
                                                           pack2<kFp16>(u[0], u[1]), pack2<kFp16>(u[2], u[3])};
        }
      }
      wave_lds_sync();
#pragma unroll
      for (int t = 0; t < 16 * kRowPieces / kWave; ++t) {
        const int r = (t * kWave + lane) / kRowPieces, c = (t * kWave + lane) % kRowPieces;
        const u32x4 bits = *reinterpret_cast<const u32x4*>(place(r, c));
        const int tr = wm * kWaveM + i * 16 + r;
        if (tile_has_row(row0, row_end, tr)) store_piece<kForm>(a, row0 + tr, col0 + wn * kWaveN + c * kPieceCols, bits);
      }
      wave_lds_sync();
    }
  } else {
    static_assert(!kGated || kNI == 4, "a pair of gate tiles and a pair of up tiles");
    float* const row_max = reinterpret_cast<float*>(sa1);  // [kWavesN][kTileM]
    uint8_t* const codes = sb0;                            // [kTileM][128], piece c of row r at c ^ r
    const int wave_col = wn * 32 + lane / 16 * 8;          // this lane's 8 columns of the block
    const bool has = col0 + wave_col < a.n;                // n is a multiple of 16
    float act[kMI][8];
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
      float m = 0.0f;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        act[i][q] = gated(acc[i][q / 4][q % 4], acc[i][2 + q / 4][q % 4]);
        m = __builtin_fmaxf(m, __builtin_fabsf(act[i][q]));
      }
      m = has ? m : 0.0f;
      m = __builtin_fmaxf(m, __shfl_xor(m, 16));
      m = __builtin_fmaxf(m, __shfl_xor(m, 32));
      if (lane < 16) row_max[wn * kTileM + wm * kWaveM + i * 16 + lane] = m;
    }
    __syncthreads();
    const int64_t block = col0 / kF8Block;
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
      const int r = wm * kWaveM + i * 16 + l16;
      float m = 0.0f;
#pragma unroll
      for (int v = 0; v < kWavesN; ++v) m = __builtin_fmaxf(m, row_max[v * kTileM + r]);
      float scale, factor;
      f8_scale(m, scale, factor);
      float f[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = act[i][q] * factor;
      *reinterpret_cast<u32x2*>(codes + r * kF8Block + (((wave_col / 16) ^ (r & 7)) * 16) + wave_col % 16) =
          u32x2{f8_pack4(f[0], f[1], f[2], f[3]), f8_pack4(f[4], f[5], f[6], f[7])};
      if (wn == 0 && lane < 16 && tile_has_row(row0, row_end, r))
        *reinterpret_cast<float*>(static_cast<uint8_t*>(a.out) + static_cast<int64_t>(row0 + r) * a.out_row_bytes +
                                  a.out_scale_off + block * 4) = scale;
    }
    __syncthreads();
    const int c = lane % 8;
    if (col0 + c * 16 >= a.n) return;
#pragma unroll
    for (int t = 0; t < kTileM / 8 / kTileWaves; ++t) {
      const int r = (t * kTileWaves + wave) * 8 + lane / 8;
      const u32x4 bits = *reinterpret_cast<const u32x4*>(codes + r * kF8Block + ((c ^ (r & 7)) * 16));
      if (tile_has_row(row0, row_end, r))
        *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.out) + static_cast<int64_t>(row0 + r) * a.out_row_bytes + col0 +
                                  c * 16) = bits;
    }
  }
}

int64_t tile_blocks(int32_t rows, int32_t groups, int32_t n, int tile_m, int tile_n) {
  return (row_slots(rows, groups, tile_m) * ((static_cast<int64_t>(n) + tile_n - 1) / tile_n) + 7) / 8 * 8;
}

template <Form kForm, bool kWide, int kTileM, int kTileN, int kWavesM>
hipError_t launch_tile(const GemmF8Args& a, hipStream_t stream) {
  constexpr int kCols = kForm == Form::kGated ? kTileN / 2 : kTileN;
  const dim3 grid(static_cast<uint32_t>(tile_blocks(a.rows, a.groups, a.n, kTileM, kCols))), block(kWave * kTileWaves);
  if (a.k % kSK != 0) tile_f8_kernel<kForm, kWide, kTileM, kTileN, kWavesM, true><<<grid, block, 0, stream>>>(a);
  else tile_f8_kernel<kForm, kWide, kTileM, kTileN, kWavesM, false><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

// One case for each kernel of select::gemm_f8_kind.
template <Form kForm>
hipError_t launch_form(const GemmF8Args& a, hipStream_t stream) {
  switch (select::gemm_f8_kind(a.rows, a.groups, a.n)) {
    case select::GemmF8Kind::kStream32: return launch_stream<kForm, 2, 4, 256>(a, stream);
    case select::GemmF8Kind::kTile64: return launch_tile<kForm, true, 64, 128, 2>(a, stream);
    case select::GemmF8Kind::kTile128: return launch_tile<kForm, true, 128, 128, 2>(a, stream);
    case select::GemmF8Kind::kTile256:
      if constexpr (kForm == Form::kF32) return launch_tile<kForm, true, 256, 128, 4>(a, stream);
      else return launch_tile<kForm, false, 256, 256, 4>(a, stream);
  }
  return hipErrorInvalidValue;
}
hipError_t launch_gated(const GemmF8Args& a, hipStream_t stream) {
  switch (select::gemm_f8_gated_kind(a.rows, a.groups, a.n)) {
    case select::GemmF8Kind::kStream32: return launch_stream<Form::kGated, 2, 8, 256>(a, stream);
    case select::GemmF8Kind::kTile64: return launch_tile<Form::kGated, true, 64, 256, 2>(a, stream);
    case select::GemmF8Kind::kTile128: return launch_tile<Form::kGated, true, 128, 256, 2>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

bool grouped_gemm_f8_fits(int32_t rows, int32_t groups, int32_t n, Form form) {
  constexpr int64_t kTileBlocks = kMaxLaunchThreads / (kTileWaves * kWave);
  if (form == Form::kGated) {
    switch (select::gemm_f8_gated_kind(rows, groups, n)) {
      case select::GemmF8Kind::kStream32: return stream_blocks(rows, groups, n, 32, 128) <= kMaxLaunchThreads / (8 * kWave);
      case select::GemmF8Kind::kTile64: return tile_blocks(rows, groups, n, 64, 128) <= kTileBlocks;
      case select::GemmF8Kind::kTile128: return tile_blocks(rows, groups, n, 128, 128) <= kTileBlocks;
      default: return false;
    }
  }
  switch (select::gemm_f8_kind(rows, groups, n)) {
    case select::GemmF8Kind::kStream32: return stream_blocks(rows, groups, n, 32, 64) <= kMaxLaunchThreads / (4 * kWave);
    case select::GemmF8Kind::kTile64: return tile_blocks(rows, groups, n, 64, 128) <= kTileBlocks;
    case select::GemmF8Kind::kTile128: return tile_blocks(rows, groups, n, 128, 128) <= kTileBlocks;
    case select::GemmF8Kind::kTile256:
      return tile_blocks(rows, groups, n, 256, form == Form::kF32 ? 128 : 256) <= kTileBlocks;
  }
  return false;
}

hipError_t launch_grouped_gemm_f8(GemmF8Args a, Form form, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  if (!grouped_gemm_f8_fits(a.rows, a.groups, a.n, form)) return hipErrorInvalidValue;
  a.nt = form != Form::kGated && select::gemm_deq_nt(a.rows, a.groups, a.k, a.n, form == Form::kF32 ? 4 : 2);
  switch (form) {
    case Form::kBf16: return launch_form<Form::kBf16>(a, stream);
    case Form::kFp16: return launch_form<Form::kFp16>(a, stream);
    case Form::kF32: return launch_form<Form::kF32>(a, stream);
    case Form::kGated: return launch_gated(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
