// Expert products in 8-bit floats: e4m3 rows times each expert's e4m3 weights,
// scaled for each 128 of a row (ts) and each 128 x 128 of the weights (ws).
// For a row m of expert g and a column j
//   y[m][j] = sum over the blocks b of k of (ts[m][b] ws[g][j / 128][b]) p_b,
//   p_b = sum over i in block b of a[m][i] w[g][j][i]
// A block's products are summed from zero by matrix instructions and added to
// the binary32 accumulator, times the block's scale, by one multiply-add.  The
// plain form rounds y; the gated form takes 2n columns, gate and up, and
// quantises g / (1 + e^-g) u in blocks of 128 columns (block_rows.h).
//
// Two matrix instructions, by what the sums become.  Where they are kept in 32
// bits (fp32 results, and the scales of 8-bit rows), the codes are widened to
// bf16 in registers: every product is exact then and the sums are binary32's
// (1.4e-7 of normal rows' results at k 7168).  The 8-bit instructions (16x16x128
// f8f6f4 at twice that rate, and 16x16x32 fp8) are not as exact: of each eight
// consecutive products they cut what lies below 2^-13 of the largest (beside
// 2^16, 2^3 is kept and 2^2 lost), 1.4e-5 of normal rows' results and at most 7 *
// 2^-13 of the largest of the eight.  They serve the tiles whose results are
// rounded to 16 bits, whose half step is 3.9e-3 (bf16) or 4.9e-4 (fp16): widened,
// 32768 rows, k 2048, n 7168 take 1050 us instead of 528, 1000 rows 67 and 63.
// split_f8_kernel, which waits for its loads, widens for every type.
//
// The weights are the first operand and the rows the second: a lane then holds
// four consecutive columns of one row, and one scale serves all four.
//
// Kernels (select_f8.h has the rule; us, at the fastest copy's 6.17 TB/s and a
// large 8-bit or bf16 library product's 3.0 and 1.25 PFLOP/s):
//
// split_f8_kernel, for the few workgroups of a small call: 16 rows and 16
// columns (and as many up columns), a quarter of k to each of four waves; the
// rows in LDS, the weights straight into registers two chunks ahead.  64 rows, k
// and n 2048, one expert: 7.7, where a tile takes 9.1.
//
// ring_f8_kernel, tiles of 32 and 64 rows by 128 rows of weights: three stages of
// 128 of k in LDS, filled by LDS-destination loads whole cache lines at a time,
// with the stage's scales in its slot.  Bound by the weights' bytes where experts
// have few rows (24 rows over 16 experts, k 2048, n 7168: 44 = 5.4 TB/s, floor
// 38), by latency where they have tens: 1000 such rows take 60 (floor 41), of
// which the last, partly filled round of workgroups is a third.  Deeper rings (four
// stages, one workgroup a CU: 64), two stages and three workgroups a CU (64),
// eight waves instead of four (59), 128 rows (80) and 256 columns were not
// faster.  The gated form's widening makes the vector ALU as busy as the matrix
// cores: 1000 rows, k 7168, n 2048, 130 (floor 77).
// As 128 x 256 it also takes the gated product of many rows, a block of 128
// columns to a workgroup, so that nothing but 8-bit rows leaves the chip: 32768
// rows 1.69-1.82 ms over boxes = 1.1 PFLOP/s, 0.9 of a large bf16 product.
//
// tile_f8_kernel, 256 x 256 by the 8-bit instruction: 32768 rows, k 2048, n 7168,
// 523-546 over boxes = 1.8 PFLOP/s.  A stage keeps the matrix cores and LDS busy for 2048
// cycles each; of a tile's 33 us, 8 find its rows, load its first stages and store
// its results with nothing else on the CU.
#include "block_rows.h"
#include "device_util.h"
#include "gemm.h"
#include "gemm_f8.h"
#include "lds_stage.h"
#include "router_util.h"
#include "row_range.h"
#include "row_slots.h"
#include "select_f8.h"
#include "select_layer.h"

#pragma clang fp contract(off)

namespace moe {
namespace {

// u g / (1 + e^-g).  Below g = -88.7 e^-g is infinite and the quotient, of at most
// 2.7e-37, becomes 0.
__device__ __forceinline__ float gated(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// Four consecutive columns of one row, as far as the row goes.
template <Form kForm>
__device__ __forceinline__ void store_columns(const GemmF8Args& a, int64_t row, int col, const f32x4& v) {
  constexpr Out kOut = kForm == Form::kAct ? Out::kF32 : static_cast<Out>(kForm);
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

// ---- few workgroups ----------------------------------------------------------------

// 16 rows and 16 columns (of the gate and of the up half).  Four waves share out
// the chunks of kSplitK of k, each with rows in LDS of its own; a lane loads its
// weights, two chunks ahead, straight into registers.  The first wave adds the
// others' sums.
constexpr int kSplitRows = 16, kSplitWaves = 4, kSplitK = 256;

template <Form kForm>
__global__ __launch_bounds__(kWave* kSplitWaves, 2) void split_f8_kernel(GemmF8Args a, int64_t slots) {
  constexpr int kHalves = kForm == Form::kAct ? 2 : 1;  // gate and up
  constexpr int kSteps = kSplitK / kF8Block, kRowPieces = kSplitK / 16;
  constexpr int kCopies = kSplitRows * kRowPieces / kWave;  // pieces of a chunk's rows that a lane brings
  constexpr int kScales = kSplitRows * kSteps;              // of a chunk, for each half
  static_assert(kRowPieces == 16 && kScales <= kWave && kF8Block % 16 == 0, "a scale a lane, one block of columns");
  constexpr int kRowsBytes = kSplitRows * kSplitK;
  __shared__ __attribute__((aligned(1024))) uint8_t rows[2][kSplitWaves][kRowsBytes];
  __shared__ float scales[2][kSplitWaves][kHalves][kScales];
  __shared__ f32x4 sums[kSplitWaves - 1][kHalves][kWave];
  const int lane = threadIdx.x % kWave, part = uniform(threadIdx.x / kWave);
  // workgroups of one block of columns lie on one XCD, an expert's slots next to each other
  const int64_t x = blockIdx.x % 8, y = blockIdx.x / 8;
  const int64_t slot = y % slots, block = y / slots * 8 + x;
  if (block * 16 >= a.n) return;
  RowSlot rs;
  if (!find_row_slot<kSplitRows>(a.group_count, a.groups, a.rows, slot, lane, &rs)) return;

  const int col0 = static_cast<int>(block) * 16;
  const int piece = lane / 16 * 16, l16 = lane % 16;
  const int kb = f8_blocks(a.k), nb = f8_blocks(a.n);
  const uint8_t* pb[kHalves];
  const float* ws[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    const int64_t half = static_cast<int64_t>(rs.group) * kHalves + h;
    pb[h] = a.w + (half * a.n + min(col0 + l16, a.n - 1)) * a.k;
    ws[h] = a.weight_scale + (half * nb + col0 / kF8Block) * kb;
  }
  const uint8_t* pa[kCopies];
  int la[kCopies];
  const int ka = lane % kRowPieces * 16;
#pragma unroll
  for (int q = 0; q < kCopies; ++q) {
    const int r = (q * kWave + lane) / kRowPieces;
    pa[q] = a.a + tile_row(rs.row0, rs.row_end, r) * a.a_stride;
    la[q] = r * kSplitK + ((lane % kRowPieces) ^ r) * 16;  // 16 rows' pieces fall into all banks
  }
  // scale `lane` of a chunk: step lane / 16, row lane % 16
  const float* pts = reinterpret_cast<const float*>(
      a.token_scale + static_cast<int64_t>(tile_row(rs.row0, rs.row_end, l16)) * a.ts_stride);
  const int rounds = (a.k + kSplitWaves * kSplitK - 1) / (kSplitWaves * kSplitK);
  // Past k the rows' codes count as zero, and so do their scales; the weights
  // there are some of the same column's.
  struct Codes {
    i32x4 a, b;
  };
  struct Rows {
    i32x4 v[kCopies];
    float s[kHalves];
  };
  auto load_a = [&](int round, Rows& to) {
    const int chunk = round * kSplitWaves + part, at = chunk * kSplitK + ka;
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      to.v[q] = *reinterpret_cast<const i32x4*>(pa[q] + (at < a.k ? at : 0));
      if (at >= a.k) to.v[q] = i32x4{0, 0, 0, 0};
    }
    const int b = chunk * kSteps + lane / kSplitRows;
    const bool have = lane < kScales && b < kb;
    const float ts = have ? pts[b] : 0.0f;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) to.s[h] = have ? ts * ws[h][b] : 0.0f;
  };
  auto put_a = [&](int buf, const Rows& from) {
#pragma unroll
    for (int q = 0; q < kCopies; ++q) *reinterpret_cast<i32x4*>(rows[buf][part] + la[q]) = from.v[q];
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
      if (lane < kScales) scales[buf][part][h][lane] = from.s[h];
  };
  auto load_b = [&](int round, Codes (&v)[kSteps][kHalves]) {
    const int chunk = round * kSplitWaves + part;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int at = chunk * kSplitK + s * kF8Block + piece;
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        v[s][h] = Codes{*reinterpret_cast<const i32x4*>(pb[h] + (at < a.k ? at : 0)),
                        *reinterpret_cast<const i32x4*>(pb[h] + (at + 64 < a.k ? at + 64 : 0))};
    }
  };
  f32x4 acc[kHalves];
#pragma unroll
  for (int h = 0; h < kHalves; ++h) acc[h] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](int buf, const Codes (&b)[kSteps][kHalves]) {
    const uint8_t* row = rows[buf][part] + l16 * kSplitK;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const WideCodes f = widen(*reinterpret_cast<const i32x4*>(row + ((s * 8 + lane / 16) ^ l16) * 16),
                                *reinterpret_cast<const i32x4*>(row + ((s * 8 + 4 + lane / 16) ^ l16) * 16));
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const f32x4 p = block_sum(widen(b[s][h].a, b[s][h].b), f);
        const float scale = scales[buf][part][h][s * kSplitRows + l16];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[h][q] = __builtin_fmaf(p[q], scale, acc[h][q]);
      }
    }
  };

  Rows a0, a1;
  Codes b0[kSteps][kHalves], b1[kSteps][kHalves];
  load_a(0, a0);
  load_b(0, b0);
  if (rounds > 1) {
    load_a(1, a1);
    load_b(1, b1);
  }
  put_a(0, a0);
  wave_lds_sync();
  // A wave's buffers are its own; it writes one again only after its reads of it.
  for (int c = 0;; c += 2) {
    multiply(0, b0);
    if (c + 1 >= rounds) break;
    if (c + 2 < rounds) {
      load_a(c + 2, a0);
      load_b(c + 2, b0);
    }
    put_a(1, a1);
    wave_lds_sync();
    multiply(1, b1);
    if (c + 2 >= rounds) break;
    if (c + 3 < rounds) {
      load_a(c + 3, a1);
      load_b(c + 3, b1);
    }
    put_a(0, a0);
    wave_lds_sync();
  }
  if (part > 0) {
#pragma unroll
    for (int h = 0; h < kHalves; ++h) sums[part - 1][h][lane] = acc[h];
  }
  __syncthreads();
  if (part > 0) return;
#pragma unroll
  for (int p = 0; p < kSplitWaves - 1; ++p)
#pragma unroll
    for (int h = 0; h < kHalves; ++h) acc[h] += sums[p][h][lane];
  if constexpr (kHalves == 2) {
#pragma unroll
    for (int q = 0; q < 4; ++q) acc[0][q] = gated(acc[0][q], acc[1][q]);
  }
  const int col = col0 + lane / 16 * 4;
  if (col < a.n && tile_has_row(rs.row0, rs.row_end, l16)) store_columns<kForm>(a, rs.row0 + l16, col, acc[0]);
}

int64_t split_blocks(int32_t rows, int32_t groups, int32_t n) {
  return row_slots(rows, groups, kSplitRows) * (((static_cast<int64_t>(n) + 15) / 16 + 7) / 8 * 8);
}

template <Form kForm>
hipError_t launch_split(const GemmF8Args& a, hipStream_t stream) {
  split_f8_kernel<kForm><<<dim3(static_cast<uint32_t>(split_blocks(a.rows, a.groups, a.n))), dim3(kWave * kSplitWaves), 0,
                           stream>>>(a, row_slots(a.rows, a.groups, kSplitRows));
  return hipGetLastError();
}

// ---- many rows for each expert -----------------------------------------------------

constexpr int kSK = kF8Block;     // bytes of k per stage: one block
constexpr int kRound = 6;         // stages of a round: the slots' places come round again
constexpr int kGroupCols = 1024;  // rows of weights of a group of column tiles

// Lane l's value is that of row l of a wave's 64 rows: in every lane, for each
// fragment i, the value of row 16 i + l % 16.
__device__ __forceinline__ void spread_rows(float v, float (&to)[4]) {
  const uint32_t b = __float_as_uint(v);
  const auto h = __builtin_amdgcn_permlane16_swap(b, b, false, false);  // rows 0 0 2 2 and 1 1 3 3
  const auto even = __builtin_amdgcn_permlane32_swap(h[0], h[0], false, false);
  const auto odd = __builtin_amdgcn_permlane32_swap(h[1], h[1], false, false);
  to[0] = __uint_as_float(even[0]), to[1] = __uint_as_float(odd[0]);
  to[2] = __uint_as_float(even[1]), to[3] = __uint_as_float(odd[1]);
}

// 16 bytes of consecutive columns of one row, as far as the row goes.
template <Form kForm>
__device__ __forceinline__ void store_piece(const GemmF8Args& a, int64_t row, int col, const u32x4& bits) {
  constexpr int kSize = kForm == Form::kF32 || kForm == Form::kAct ? 4 : 2, kCols = 16 / kSize;
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
      if constexpr (kSize == 4) static_cast<uint32_t*>(a.out)[at + q] = bits[q];
      else static_cast<uint16_t*>(a.out)[at + q] = static_cast<uint16_t>(bits[q / 2] >> (q % 2 * 16));
    }
  }
}

// What every wave of a tile knows: the tile's rows and columns, its share of
// the loads, and where its scales stand.
//
// Tiles in order: groups of column tiles, the row slots of a group, its
// columns; XCD x (workgroups x, x + 8, ...) takes the x-th eighth of the tiles
// that the counts give.
template <Form kForm, int kTileM, int kTileN, int kWavesM, int kWavesN_>
struct TileWave {
  static constexpr bool kGated = kForm == Form::kGated || kForm == Form::kAct;
  static constexpr int kHalves = kGated ? 2 : 1;  // gate and up
  static constexpr int kWavesN = kWavesN_, kTileWaves = kWavesM * kWavesN;
  static constexpr int kWaveM = kTileM / kWavesM, kWaveN = kTileN / kWavesN;
  static constexpr int kMI = kWaveM / 16, kNI = kWaveN / 16;
  static constexpr int kCols = kTileN / kHalves;  // columns of the result
  static constexpr int kRowsPerLoad = kWave / (kSK / 16);
  static constexpr int kLoadsA = kTileM / kRowsPerLoad / kTileWaves, kLoadsB = kTileN / kRowsPerLoad / kTileWaves;
  static_assert(kTileWaves % 2 == 0 && kWaveM % 32 == 0, "what the swizzles go by");
  static_assert(kF8Block % (kWaveN / kHalves) == 0 && (kForm != Form::kGated || kCols == kF8Block) &&
                    kWaveN / kHalves % 32 == 0,
                "a wave's columns share a scale, and fall into pairs of fragments");

  int lane, wave, wm, wn, l16, row0, row_end, col0, stages, start;
  // Load q of a wave fills the stage rows from 8 (q kTileWaves + wave); lane l
  // fetches the piece that belongs at position l % 8 of row l / 8.  A wave's stage
  // rows of weights are its gate rows, then its up rows.  Offsets from the tile's first row fit in 32 bits: 256 rows of at most
  // kF8MaxRowBytes, and weights of at most 2^16 columns by 2^16 with 256 more.
  int piece, k;  // (the piece of load 0)
  // kTileWaves is even: q turns the bit of swizzle() that rows 16 apart differ in.
  __device__ __forceinline__ int piece_of(int q) const { return piece ^ ((q * (kTileWaves / 2) & 1) << 1); }
  // The tile of 256 x 256 has no registers left for its loads' offsets and makes
  // them anew each time, of the last row (of weights) that exists and the stride.
  static constexpr bool kAnew = kTileM * kTileN == 256 * 256;
  static constexpr bool kTurned = kTileM <= 64;  // (larger tiles are not bound by their loads)
  const uint8_t *base_a, *base_b;
  uint32_t src_a[kAnew ? 1 : kLoadsA], src_b[kAnew ? 1 : kLoadsB];
  int last_a, last_b;
  uint32_t stride_a;
  const float* ts_row;        // the scales of the wave's row lane % kWaveM
  const float* ws[kHalves];   // of its columns
  // Fragments: pair p, tile t of the weights is row 32 p + 8 (l16 / 4) + 4 t +
  // l16 % 4, so that a lane ends with 8 consecutive columns in the two tiles.
  int frag_a, frag_b, swz_a, swz_b;

  __device__ __forceinline__ bool set(const GemmF8Args& a) {
    lane = threadIdx.x % kWave, wave = uniform(threadIdx.x / kWave);
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
    if (!place_row_slot<kTileM>(a.group_count, a.groups, a.rows, lane, pick, &rs)) return false;
    row0 = rs.row0, row_end = rs.row_end;
    col0 = static_cast<int>(col_tile) * kCols;
    wm = wave / kWavesN, wn = wave % kWavesN, l16 = lane % 16;
    stages = f8_blocks(a.k), k = a.k;
    // Where along k the stages begin.  Rows that lie a multiple of 4096 bytes apart
    // fall into few memory channels, and workgroups in step would all ask the same
    // ones (16 experts, us, all from 0 and each expert from a place of its own: k
    // and n 4096, 24 rows 65.1 and 46.0, 1000 rows 70.8, 67.4; k 8192, n 2048, 24
    // rows 60.8, 45.3; gated, k 4096, n 2048, 24 rows 69.4, 50.6).
    start = !kTurned || a.k % 4096 != 0 ? 0 : static_cast<int>(rs.group * int64_t(5) % stages);
    piece = (lane % 8) ^ swizzle(kRowsPerLoad * wave + lane / 8);
    base_a = a.a + row0 * a.a_stride;
    base_b = a.w + (static_cast<int64_t>(rs.group) * kHalves * a.n + col0) * a.k;
    last_a = row_end - row0 - 1, last_b = a.n - 1 - col0, stride_a = static_cast<uint32_t>(a.a_stride);
#pragma unroll
    for (int q = 0; q < (kAnew ? 0 : kLoadsA); ++q) {
      const int r = kRowsPerLoad * (q * kTileWaves + wave) + lane / 8;
      src_a[q] = static_cast<uint32_t>(tile_row(row0, row_end, r) - row0) * stride_a + piece_of(q) * 16;
    }
#pragma unroll
    for (int q = 0; q < (kAnew ? 0 : kLoadsB); ++q) {
      const int r = kRowsPerLoad * (q * kTileWaves + wave) + lane / 8;
      constexpr int kPart = kWaveN / kHalves;
      const int half = r % kWaveN / kPart, c = r / kWaveN * kPart + r % kPart;
      src_b[q] = static_cast<uint32_t>(half * a.n + min(c, a.n - 1 - col0)) * static_cast<uint32_t>(a.k) + piece_of(q) * 16;
    }
    ts_row = reinterpret_cast<const float*>(
        a.token_scale + static_cast<int64_t>(tile_row(row0, row_end, wm * kWaveM + lane % kWaveM)) * a.ts_stride);
    const int nb = f8_blocks(a.n);
    const int col_block = uniform(min((col0 + wn * (kWaveN / kHalves)) / kF8Block, nb - 1));
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
      ws[h] = a.weight_scale + ((static_cast<int64_t>(rs.group) * kHalves + h) * nb + col_block) * stages;
    frag_a = (wm * kWaveM + l16) * kSK;
    const int row_b = 8 * (l16 / 4) + l16 % 4;
    frag_b = (wn * kWaveN + row_b) * kSK;
    swz_a = swizzle(l16), swz_b = swizzle(row_b);
    return true;
  }

  // The block of k of stage s; stages past the last one repeat it.
  __device__ __forceinline__ int block_of(int s) const {
    s = min(s, stages - 1);
    return !kTurned || s + start < stages ? s + start : s + start - stages;
  }
  // Stages past the last one load it again, into slots that are not read; a
  // piece past k reads the row's first piece (its row fragments count as zero).
  template <bool kTail, int kLoads>
  __device__ __forceinline__ void issue(int s, const uint8_t* base, const uint32_t* src, int last, uint32_t stride,
                                        uint8_t* buf) const {
    const int k0 = block_of(s) * kSK;
    int first = kRowsPerLoad * wave + lane / 8;
    if constexpr (kAnew) asm volatile("" : "+v"(first));  // else the offsets are made once and kept
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      uint32_t at;
      if constexpr (kAnew)
        at = static_cast<uint32_t>(min(kRowsPerLoad * kTileWaves * q + first, last)) * stride + piece_of(q) * 16;
      else at = src[q];
      const uint8_t* p;
      if constexpr (kTail) p = base + (at + static_cast<uint32_t>((k0 + piece_of(q) * 16 < k) ? k0 : -piece_of(q) * 16));
      else p = base + k0 + at;
      __builtin_amdgcn_global_load_lds(p, (MOE_LDS void*)(buf + (q * kTileWaves + wave) * kRowsPerLoad * kSK), 16, 0, 0);
    }
  }
  template <bool kTail>
  __device__ __forceinline__ void issue_a(int s, uint8_t* buf) const {
    issue<kTail, kLoadsA>(s, base_a, src_a, last_a, stride_a, buf);
  }
  template <bool kTail>
  __device__ __forceinline__ void issue_b(int s, uint8_t* buf) const {
    issue<kTail, kLoadsB>(s, base_b, src_b, last_b, static_cast<uint32_t>(k), buf);
  }
  // The two pieces of fragment i of a stage's rows, and j of its weights.
  __device__ __forceinline__ void read_a(const uint8_t* buf, int i, i32x4 (&to)[2]) const {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      to[q] = *reinterpret_cast<const i32x4*>(buf + frag_a + i * 16 * kSK +
                                              ((4 * q + lane / 16) ^ swz_a ^ ((i & 1) << 1)) * 16);
  }
  __device__ __forceinline__ void read_b(const uint8_t* buf, int j, i32x4 (&to)[2]) const {
#pragma unroll
    for (int q = 0; q < 2; ++q)
      to[q] = *reinterpret_cast<const i32x4*>(buf + frag_b + ((j >> 1) * 32 + (j & 1) * 4) * kSK +
                                              ((4 * q + lane / 16) ^ swz_b ^ ((j & 1) << 1)) * 16);
  }
  // Zeros for a row fragment's pieces past k, in stage s.
  __device__ __forceinline__ void cut_tail(int s, i32x4 (&a)[2]) const {
#pragma unroll
    for (int q = 0; q < 2; ++q) a[q] &= s * kSK + (4 * q + lane / 16) * 16 < k ? -1 : 0;
  }
};

// A tile's results.  They pass through LDS, so that a store's lanes lie along
// rows (whole cache lines): `lds0` and `lds1` of kTileN stage rows each, and
// `small` for the row maxima.
template <Form kForm, int kTileM, int kTileN, int kWavesM, int kWavesN, int kMI, int kNI>
__device__ __forceinline__ void store_tile(const GemmF8Args& a,
                                           const TileWave<kForm, kTileM, kTileN, kWavesM, kWavesN>& t,
                                           const f32x4 (&acc)[kMI][kNI], uint8_t* lds0, uint8_t* lds1,
                                           uint8_t* small) {
  using T = TileWave<kForm, kTileM, kTileN, kWavesM, kWavesN>;
  constexpr int kWaveM = T::kWaveM, kWaveN = T::kWaveN, kTileWaves = T::kTileWaves;
  const int lane = t.lane, wave = t.wave, l16 = t.l16, wm = t.wm, wn = t.wn, col0 = t.col0;
  const int row0 = t.row0, row_end = t.row_end;
  if constexpr (kForm != Form::kGated) {
    constexpr bool kFloats = kForm == Form::kF32 || kForm == Form::kAct;
    constexpr int kPieceCols = kFloats ? 4 : 8;       // columns of a 16-byte piece
    constexpr int kWaveCols = kWaveN / T::kHalves;  // of the result
    constexpr int kRowPieces = kWaveCols / kPieceCols, kWaveBytes = 16 * kRowPieces * 16;
    constexpr int kSlotWaves = kTileN * kSK / kWaveBytes < kTileWaves ? kTileN * kSK / kWaveBytes : kTileWaves;
    static_assert(2 * kSlotWaves >= kTileWaves, "two slots hold every wave's rows");
    uint8_t* const mine = (wave < kSlotWaves ? lds0 : lds1) + wave % kSlotWaves * kWaveBytes;
    // piece c of row r lies at c ^ r, so that 16 rows' pieces fall into all banks
    constexpr int kTurn = (kRowPieces < 16 ? kRowPieces : 16) - 1;
    const auto place = [&](int r, int c) { return mine + (r * kRowPieces + (c ^ (r & kTurn))) * 16; };
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
#pragma unroll
      for (int p = 0; p < kNI / 2 / T::kHalves; ++p) {
        f32x4 v = acc[i][2 * p], u = acc[i][2 * p + 1];
        if constexpr (kForm == Form::kAct) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            v[q] = gated(v[q], acc[i][kNI / 2 + 2 * p][q]);
            u[q] = gated(u[q], acc[i][kNI / 2 + 2 * p + 1][q]);
          }
        }
        const int c = (p * 4 + lane / 16) * (8 / kPieceCols);
        if constexpr (kFloats) {
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
      for (int x = 0; x < 16 * kRowPieces / kWave; ++x) {
        const int r = (x * kWave + lane) / kRowPieces, c = (x * kWave + lane) % kRowPieces;
        const u32x4 bits = *reinterpret_cast<const u32x4*>(place(r, c));
        const int tr = wm * kWaveM + i * 16 + r;
        if (tile_has_row(row0, row_end, tr))
          store_piece<kForm>(a, row0 + tr, col0 + wn * kWaveCols + c * kPieceCols, bits);
      }
      wave_lds_sync();
    }
  } else {
    static_assert(kForm != Form::kGated || kNI == 4, "a pair of gate tiles and a pair of up tiles");
    float* const row_max = reinterpret_cast<float*>(small);  // [kWavesN][kTileM]
    uint8_t* const codes = lds0;                            // [kTileM][128], piece c of row r at c ^ r
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
    for (int x = 0; x < kTileM / 8 / kTileWaves; ++x) {
      const int r = (x * kTileWaves + wave) * 8 + lane / 8;
      const u32x4 bits = *reinterpret_cast<const u32x4*>(codes + r * kF8Block + ((c ^ (r & 7)) * 16));
      if (tile_has_row(row0, row_end, r))
        *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(a.out) + static_cast<int64_t>(row0 + r) * a.out_row_bytes + col0 +
                                  c * 16) = bits;
    }
  }
}

// The 8-bit instruction: eight waves in two groups, one wave of each per SIMD,
// half a step apart; while one multiplies, the other reads its fragments.
template <Form kForm, int kTileM, int kTileN, int kWavesM, int kWavesN, bool kTail>
__global__ __launch_bounds__(kWave* kWavesM* kWavesN) void tile_f8_kernel(GemmF8Args a) {
  using T = TileWave<kForm, kTileM, kTileN, kWavesM, kWavesN>;
  static_assert(T::kTileWaves == 8, "two groups of four waves");
  constexpr int kMI = T::kMI, kNI = T::kNI, kStepNI = kNI / 2;
  __shared__ __attribute__((aligned(1024))) uint8_t sa0[kTileM * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sa1[kTileM * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sb0[kTileN * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sb1[kTileN * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sb2[kTileN * kSK];
  T t;
  if (!t.set(a)) return;  // the whole workgroup
  const int stages = t.stages;
  // The scales: lane l has those of the wave's row l, two stages ahead.  The
  // weights' are the same for all rows; lane l has the one l stages on, a round
  // ahead.  (As scalar loads they made every wait for LDS wait for memory.)
  float row_scale[2], col_scales, next_col_scales;
  const auto load_col_scales = [&](int first) { return t.ws[0][min(first + t.lane, stages - 1)]; };
  f32x4 acc[kMI][kNI];
#pragma unroll
  for (int i = 0; i < kMI; ++i)
#pragma unroll
    for (int j = 0; j < kNI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  i32x8 af[kMI];
  // Half of a stage's columns.
  auto step = [&](int S, int h, float ts, float w, const uint8_t* ca, const uint8_t* cb, uint8_t* fill_a,
                  uint8_t* fill_b) {
    if (h == 0) t.template issue_a<kTail>(S + 1, fill_a);  // into the slot A(S - 1) used
    else t.template issue_b<kTail>(S + 2, fill_b);         // into the slot B(S - 1) used
    i32x4 ra[kMI][2], rb[kStepNI][2];
    if (h == 0) {
#pragma unroll
      for (int i = 0; i < kMI; ++i) t.read_a(ca, i, ra[i]);
    }
#pragma unroll
    for (int n = 0; n < kStepNI; ++n) t.read_b(cb, h * kStepNI + n, rb[n]);
    float s[kMI];
    spread_rows(ts, s);
#pragma unroll
    for (int i = 0; i < kMI; ++i) s[i] *= w;
    // this wave's loads of A(S + 1) and B(S + 1); those of B(S + 2) may still run
    if (h == 1) __builtin_amdgcn_s_waitcnt(vmcnt_wait(T::kLoadsB));
    __builtin_amdgcn_s_waitcnt(kLgkmWait0);
    if (h == 0) {
#pragma unroll
      for (int i = 0; i < kMI; ++i) {
        if constexpr (kTail) t.cut_tail(S, ra[i]);
        af[i] = join(ra[i][0], ra[i][1]);
      }
    }
    tile_barrier();
#pragma unroll
    for (int n = 0; n < kStepNI; ++n) {
      f32x4 part[kMI];
#pragma unroll
      for (int i = 0; i < kMI; ++i) part[i] = block_sum(join(rb[n][0], rb[n][1]), af[i]);
#pragma unroll
      for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[i][h * kStepNI + n][q] = __builtin_fmaf(part[i][q], s[i], acc[i][h * kStepNI + n][q]);
    }
    tile_barrier();
  };
  auto stage = [&](int S, int u, const uint8_t* ca, const uint8_t* cb, uint8_t* fill_a, uint8_t* fill_b) {
    const float w = lane_float(col_scales, u);
    step(S, 0, row_scale[u % 2], w, ca, cb, fill_a, fill_b);
    step(S, 1, row_scale[u % 2], w, ca, cb, fill_a, fill_b);
    row_scale[u % 2] = t.ts_row[min(S + 2, stages - 1)];
  };
  next_col_scales = load_col_scales(0);
#pragma unroll
  for (int u = 0; u < 2; ++u) row_scale[u] = t.ts_row[min(u, stages - 1)];
  t.template issue_b<kTail>(0, sb0);
  t.template issue_a<kTail>(0, sa0);
  t.template issue_b<kTail>(1, sb1);
  __builtin_amdgcn_s_waitcnt(vmcnt_wait(T::kLoadsB));
  tile_barrier();
  const int grp = t.wave / 4;
  if (grp == 1) tile_barrier();  // the second group runs half a step behind
  const int rounds = stages / kRound;
  for (int r = 0; r < rounds; ++r) {
    col_scales = next_col_scales;
    next_col_scales = load_col_scales(kRound * (r + 1));
    stage(kRound * r, 0, sa0, sb0, sa1, sb2);
    stage(kRound * r + 1, 1, sa1, sb1, sa0, sb0);
    stage(kRound * r + 2, 2, sa0, sb2, sa1, sb1);
    stage(kRound * r + 3, 3, sa1, sb0, sa0, sb2);
    stage(kRound * r + 4, 4, sa0, sb1, sa1, sb0);
    stage(kRound * r + 5, 5, sa1, sb2, sa0, sb1);
  }
  {
    col_scales = next_col_scales;
    const int rest = stages - rounds * kRound;
    if (rest > 0) stage(kRound * rounds, 0, sa0, sb0, sa1, sb2);
    if (rest > 1) stage(kRound * rounds + 1, 1, sa1, sb1, sa0, sb0);
    if (rest > 2) stage(kRound * rounds + 2, 2, sa0, sb2, sa1, sb1);
    if (rest > 3) stage(kRound * rounds + 3, 3, sa1, sb0, sa0, sb2);
    if (rest > 4) stage(kRound * rounds + 4, 4, sa0, sb1, sa1, sb0);
  }
  if (grp == 0) tile_barrier();  // every wave passes the same number of barriers
  // no load may still be writing this workgroup's LDS, and no wave reading it
  __builtin_amdgcn_s_waitcnt(vmcnt_wait(0));
  tile_barrier();
  store_tile(a, t, acc, sb0, sb1, sa1);
}

// A ring of three stages in LDS, of which one is multiplied while the others'
// loads run; the waves meet once a stage.  For the widened codes the vector ALU
// has nearly as much to do as the matrix cores (16 conversions a fragment, 4
// multiply-adds for each 4 matrix instructions), and overlaps with them freely.
template <bool kWide>
struct FragmentOf {
  using Type = i32x8;
  static __device__ __forceinline__ Type make(const i32x4 (&r)[2]) { return join(r[0], r[1]); }
};
template <>
struct FragmentOf<true> {
  using Type = WideCodes;
  static __device__ __forceinline__ Type make(const i32x4 (&r)[2]) { return widen(r[0], r[1]); }
};

template <Form kForm, bool kWide, int kTileM, int kTileN, int kWavesM, int kWavesN, bool kTail>
__global__ __launch_bounds__(kWave* kWavesM* kWavesN, 2) void ring_f8_kernel(GemmF8Args a) {
  using T = TileWave<kForm, kTileM, kTileN, kWavesM, kWavesN>;
  using F = FragmentOf<kWide>;
  constexpr int kMI = T::kMI, kNI = T::kNI, kSlots = 3;
  __shared__ __attribute__((aligned(1024))) uint8_t sa0[kTileM * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sa1[kTileM * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sa2[kTileM * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sb0[kTileN * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sb1[kTileN * kSK];
  __shared__ __attribute__((aligned(1024))) uint8_t sb2[kTileN * kSK];
  constexpr int kScaleFloats = (kTileM + kWave - 1) / kWave * kWave + kWave;
  __shared__ float ss0[kScaleFloats], ss1[kScaleFloats], ss2[kScaleFloats];
  T t;
  if (!t.set(a)) return;  // the whole workgroup
  const int stages = t.stages;
  f32x4 acc[kMI][kNI];
#pragma unroll
  for (int i = 0; i < kMI; ++i)
#pragma unroll
    for (int j = 0; j < kNI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  // A stage's scales lie in its slot, brought by one load of each wave: the
  // first waves have 64 rows each, the others all the same one or two of the
  // weights (a tile's columns lie in one block).  Loaded into registers by each
  // wave for itself, the rows' with a vector and the weights' with a scalar load,
  // they cost 1000 rows, k 2048, n 7168 7 and 14 of 75 us.
  constexpr int kLoads = T::kLoadsA + T::kLoadsB + 1, kRowWaves = (kTileM + kWave - 1) / kWave;
  static_assert(kRowWaves < T::kTileWaves, "a wave for the weights' scales");
  const float* scale_src;
  if (t.wave < kRowWaves) {
    scale_src = reinterpret_cast<const float*>(
        a.token_scale + static_cast<int64_t>(tile_row(t.row0, t.row_end, min(t.wave * kWave + t.lane, kTileM - 1))) * a.ts_stride);
  } else {
    scale_src = t.lane % T::kHalves == 0 ? t.ws[0] : t.ws[T::kHalves - 1];
  }
  const int scale_at = t.wave < kRowWaves ? t.wave * kWave : kRowWaves * kWave;
  const auto issue = [&](int S, uint8_t* to_a, uint8_t* to_b, float* to_s) {
    t.template issue_b<kTail>(S, to_b);
    t.template issue_a<kTail>(S, to_a);
    __builtin_amdgcn_global_load_lds(scale_src + t.block_of(S), (MOE_LDS void*)(to_s + scale_at), 4, 0, 0);
  };
  issue(0, sa0, sb0, ss0);
  issue(1, sa1, sb1, ss1);
  __builtin_amdgcn_s_waitcnt(vmcnt_wait((kSlots - 2) * kLoads));
  tile_barrier();
  auto stage = [&](int S, const uint8_t* ca, const uint8_t* cb, const float* cs, uint8_t* fill_a, uint8_t* fill_b,
                   float* fill_s) {
    issue(S + kSlots - 1, fill_a, fill_b, fill_s);  // into the slot of stage S - 1
    i32x4 ra[kMI][2], rb[2][2];
#pragma unroll
    for (int i = 0; i < kMI; ++i) t.read_a(ca, i, ra[i]);
    t.read_b(cb, 0, rb[0]);
    float row[kMI], ws[T::kHalves];
#pragma unroll
    for (int i = 0; i < kMI; ++i) row[i] = cs[t.wm * T::kWaveM + i * 16 + t.l16];
#pragma unroll
    for (int h = 0; h < T::kHalves; ++h) ws[h] = cs[kRowWaves * kWave + h];
    typename F::Type af[kMI];
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
      if constexpr (kTail) t.cut_tail(S, ra[i]);
      af[i] = F::make(ra[i]);
    }
    // The next fragment is read, and the last one's sums join, while a fragment
    // is multiplied.
    f32x4 p[2][kMI];
    const auto join_sums = [&](int j) {
#pragma unroll
      for (int i = 0; i < kMI; ++i) {
        const float s = row[i] * ws[j / (kNI / T::kHalves)];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i][j][q] = __builtin_fmaf(p[j % 2][i][q], s, acc[i][j][q]);
      }
    };
#pragma unroll
    for (int j = 0; j < kNI; ++j) {
      if (j + 1 < kNI) t.read_b(cb, j + 1, rb[(j + 1) % 2]);
      const typename F::Type bf = F::make(rb[j % 2]);
      if constexpr (kWide) {
#pragma unroll
        for (int i = 0; i < kMI; ++i) p[j % 2][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int i = 0; i < kMI; ++i)
            p[j % 2][i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf.v[q], af[i].v[q], p[j % 2][i], 0, 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < kMI; ++i) p[j % 2][i] = block_sum(bf, af[i]);
      }
      if (j > 0) join_sums(j - 1);
    }
    join_sums(kNI - 1);
    // this wave's loads of stage S + 1, and its reads of stage S
    __builtin_amdgcn_s_waitcnt(vmcnt_wait((kSlots - 2) * kLoads));
    __builtin_amdgcn_s_waitcnt(kLgkmWait0);
    tile_barrier();
  };
  const int rounds = stages / kSlots, rest = stages - rounds * kSlots;
  int S = 0;
  for (int r = 0; r < rounds; ++r, S += 3) {
    stage(S, sa0, sb0, ss0, sa2, sb2, ss2);
    stage(S + 1, sa1, sb1, ss1, sa0, sb0, ss0);
    stage(S + 2, sa2, sb2, ss2, sa1, sb1, ss1);
  }
  if (rest > 0) stage(S, sa0, sb0, ss0, sa2, sb2, ss2);
  if (rest > 1) stage(S + 1, sa1, sb1, ss1, sa0, sb0, ss0);
  // no load may still be writing this workgroup's LDS
  __builtin_amdgcn_s_waitcnt(vmcnt_wait(0));
  tile_barrier();
  store_tile(a, t, acc, sb0, sb1, sa1);
}

int64_t tile_blocks(int32_t rows, int32_t groups, int32_t n, int tile_m, int tile_n) {
  return (row_slots(rows, groups, tile_m) * ((static_cast<int64_t>(n) + tile_n - 1) / tile_n) + 7) / 8 * 8;
}

constexpr int tile_cols(Form form, int tile_n) {
  return form == Form::kGated || form == Form::kAct ? tile_n / 2 : tile_n;
}

template <Form kForm, int kTileM, int kTileN, int kWavesM, int kWavesN>
hipError_t launch_tile(const GemmF8Args& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(tile_blocks(a.rows, a.groups, a.n, kTileM, tile_cols(kForm, kTileN))));
  const dim3 block(kWave * kWavesM * kWavesN);
  if (a.k % kSK != 0) tile_f8_kernel<kForm, kTileM, kTileN, kWavesM, kWavesN, true><<<grid, block, 0, stream>>>(a);
  else tile_f8_kernel<kForm, kTileM, kTileN, kWavesM, kWavesN, false><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}
template <Form kForm, bool kWide, int kTileM, int kTileN, int kWavesM, int kWavesN>
hipError_t launch_ring(const GemmF8Args& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(tile_blocks(a.rows, a.groups, a.n, kTileM, tile_cols(kForm, kTileN))));
  const dim3 block(kWave * kWavesM * kWavesN);
  if (a.k % kSK != 0)
    ring_f8_kernel<kForm, kWide, kTileM, kTileN, kWavesM, kWavesN, true><<<grid, block, 0, stream>>>(a);
  else
    ring_f8_kernel<kForm, kWide, kTileM, kTileN, kWavesM, kWavesN, false><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

// One case for each kernel of select::gemm_f8_kind.
template <Form kForm>
hipError_t launch_form(const GemmF8Args& a, hipStream_t stream) {
  constexpr bool kWide = kForm == Form::kF32;
  switch (select::gemm_f8_kind(a.rows, a.groups, a.n, kWide)) {
    case select::GemmF8Kind::kSplit16: return launch_split<kForm>(a, stream);
    case select::GemmF8Kind::kTile32: return launch_ring<kForm, kWide, 32, 128, 1, 2>(a, stream);
    case select::GemmF8Kind::kTile64: return launch_ring<kForm, kWide, 64, 128, 2, 2>(a, stream);
    case select::GemmF8Kind::kTile256:
      if constexpr (kWide) return launch_ring<kForm, true, 256, 128, 4, 2>(a, stream);
      else return launch_tile<kForm, 256, 256, 4, 2>(a, stream);
  }
  return hipErrorInvalidValue;
}
hipError_t launch_act(const GemmF8Args& a, hipStream_t stream) {
  switch (select::gemm_f8_act_kind(a.rows, a.groups, a.n)) {
    case select::GemmF8Kind::kSplit16: return launch_split<Form::kAct>(a, stream);
    case select::GemmF8Kind::kTile32: return launch_ring<Form::kAct, true, 32, 128, 1, 2>(a, stream);
    case select::GemmF8Kind::kTile64: return launch_ring<Form::kAct, true, 64, 128, 2, 2>(a, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

// The workspace's rows of activations, quantised: 16 lanes a block of 128
// columns, four blocks a wave.  Rows that no expert owns are not read.
__global__ __launch_bounds__(256) void quant_act_f8_kernel(GemmF8Args a, const float* act, int64_t items) {
  const int lane = threadIdx.x % kWave;
  const int quads = (f8_blocks(a.n) + 3) / 4;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + uniform(threadIdx.x / kWave);
  if (item >= items) return;
  const int64_t row = item / quads;
  uint32_t owned = 0;  // rows of the experts, whose sum may pass 2^32: a sum that saturates is past `rows`
  for (int g = lane; g < a.groups; g += kWave) owned = add_sat(owned, static_cast<uint32_t>(max(a.group_count[g], 0)));
  for (int d = 1; d < kWave; d *= 2) owned = add_sat(owned, static_cast<uint32_t>(__shfl_xor(static_cast<int>(owned), d)));
  if (row >= owned) return;
  const int block = static_cast<int>(item % quads) * 4 + lane / 16, col = block * kF8Block + lane % 16 * 8;
  const bool has = col < a.n;  // n is a multiple of 16
  float f[8], m = 0.0f;
  const f32x4* src = reinterpret_cast<const f32x4*>(act + row * a.n + (has ? col : 0));
  const f32x4 u = src[0], v = src[1];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    f[q] = q < 4 ? u[q % 4] : v[q % 4];
    m = __builtin_fmaxf(m, __builtin_fabsf(f[q]));
  }
  float scale, factor;
  f8_scale(token_max<16>(has ? m : 0.0f), scale, factor);
  if (!has) return;
  uint8_t* dst = static_cast<uint8_t*>(a.out) + row * a.out_row_bytes;
#pragma unroll
  for (int q = 0; q < 8; ++q) f[q] *= factor;
  *reinterpret_cast<u32x2*>(dst + col) = u32x2{f8_pack4(f[0], f[1], f[2], f[3]), f8_pack4(f[4], f[5], f[6], f[7])};
  if (lane % 16 == 0) *reinterpret_cast<float*>(dst + a.out_scale_off + block * 4) = scale;
}

bool grouped_gemm_f8_fits(int32_t rows, int32_t groups, int32_t n, Form form) {
  const auto split = [&]() { return split_blocks(rows, groups, n) <= kMaxLaunchThreads / (kSplitWaves * kWave); };
  const auto tile = [&](int tile_m, int tile_n, int waves) {
    return tile_blocks(rows, groups, n, tile_m, tile_n) <= kMaxLaunchThreads / (waves * kWave);
  };
  if (form == Form::kGated) {
    if (!select::gemm_f8_act(rows, groups, n)) return tile(128, 128, 8);
    switch (select::gemm_f8_act_kind(rows, groups, n)) {
      case select::GemmF8Kind::kSplit16: return split();
      case select::GemmF8Kind::kTile32: return tile(32, 64, 2);
      case select::GemmF8Kind::kTile64: return tile(64, 64, 4);
      default: return false;
    }
  }
  switch (select::gemm_f8_kind(rows, groups, n, form == Form::kF32)) {
    case select::GemmF8Kind::kSplit16: return split();
    case select::GemmF8Kind::kTile32: return tile(32, 128, 2);
    case select::GemmF8Kind::kTile64: return tile(64, 128, 4);
    case select::GemmF8Kind::kTile256: return tile(256, form == Form::kF32 ? 128 : 256, 8);
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
    default: break;
  }
  if (!select::gemm_f8_act(a.rows, a.groups, a.n)) return launch_ring<Form::kGated, true, 128, 256, 2, 4>(a, stream);
  GemmF8Args first = a;
  first.out = a.workspace;
  const hipError_t e = launch_act(first, stream);
  if (e != hipSuccess) return e;
  const int64_t items = static_cast<int64_t>(a.rows) * ((f8_blocks(a.n) + 3) / 4);
  quant_act_f8_kernel<<<dim3(static_cast<uint32_t>((items + 3) / 4)), dim3(4 * kWave), 0, stream>>>(
      a, static_cast<const float*>(a.workspace), items);
  return hipGetLastError();
}

}  // namespace moe
