// Second expert matmul of the MoE layer's expert side (GMM2): int8 rows times
// each expert's int8 weights, scaled by token and by output channel
// ("UMDK/CAM communication acceleration library deep analysis v2", section
// 4.3).  For a row m of expert g and a column j
//   out[m][j] = round((float(sum_i a[m][i] w[g][j][i]) * ws[g][j]) * ts_m)
// with the sum exact in int32 (below 2^31 for any order) and each later
// operation rounded to binary32, so the result does not depend on the tiling.
//
// The weights are the first operand of v_mfma_i32_16x16x64_i8 and the rows
// the second: a lane then holds four consecutive columns of one row, which it
// scales with one token scale and stores together.
//
// Two kernels (select_layer.h has the rule):
//
// stream_kernel, for experts with few rows, where the weights' bytes are the
// work: a workgroup takes kMI x 16 rows and 64 columns, or 32 and two parts of
// k.  The rows lie in LDS in chunks of kKC bytes of k, two buffers; a wave owns
// 16 columns and loads their weights straight into registers, two chunks ahead,
// each byte once.  (A fragment load touches 16 rows at 64 bytes each; with the
// rows' fragments loaded that way too, a decode step took 50 us instead of 44.)
// 24 rows over 16 experts, k 2048, n 7168: 43 us = 5.5 TB/s, nearly all of it
// reads.  Where such workgroups would leave most CUs idle, one
// takes 16 columns only and its four waves a quarter of k each (64 rows over 8
// experts, k 4096, n 1024: 8.9 us instead of 12.4; the same split within 64
// columns, 12.8: a CU's loads in flight are the limit there, not the chain of
// chunks).
//
// tile_kernel, for experts with more rows: eight waves in two groups, one wave
// of each per SIMD, half a step apart; while one multiplies, the other reads
// its fragments.  K is walked in stages of 128 bytes that the LDS-destination
// loads fill, whole cache lines (two slots for the rows, three for the
// weights); the schedule is that of the first expert matmul (gemm.hip), with
// its reasons.  The tiles of 64 x 128 and 128 x 128 take at most 80 KB of LDS,
// so two workgroups share a CU and one's start and stores run under the
// other's products; the tile of 256 x 256 takes all of it and moves half the
// bytes from L2 per product.  Results pass through LDS to whole cache lines.
// Tiles are dealt to the XCDs by the number that the counts give, not by the
// launch's bound: an eighth each, in an order in which an XCD's L2 holds the
// weights of 1024 columns while the rows pass.  (Dealt by the bound, XCDs with
// empty slots idled: 16384 rows over 64 experts, k and n 2048, took 132 us
// instead of 112.)  1000 rows over 16 experts, k 2048, n 7168: 53 us = 4.7 TB/s.
// 32768 rows: 460 us = 2.09 POP/s (a large library product: 2.12).  A tile there takes 33 us: 3 to find its rows and load its first
// stages, 24 for 16 stages, 5 for its results.  A stage keeps the matrix cores
// busy for 2048 cycles and LDS too (192 KB of fragments, 64 KB of loads at 128
// bytes a cycle), 17 us of the 24 at the clock that the chip holds under this
// load; they do not overlap fully.  Not faster: one resident workgroup a CU
// that loads the next tile's first stages before it stores (511 and 486 us), four
// waves of 128 x 128 (550, 489), weight fragments read a step ahead (the same;
// the masked instance of 128 x 128 spills), loads left out past the last stage
// (the accumulators spill where the paths meet), token scales loaded before the
// loop, groups of 512 columns; groups of 2048 are 7 % slower.
#include "device_util.h"
#include "gemm.h"
#include "layer.h"
#include "router_util.h"
#include "row_range.h"
#include "row_slots.h"

#pragma clang fp contract(off)

namespace moe {
namespace {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
#define MOE_LDS __attribute__((address_space(3)))

// Stores below are at any element's address: one unaligned store of 16 bytes
// costs far less than eight stores.

// Where along k a workgroup begins (the sums are exact in any order).  Rows that
// lie a multiple of 4096 bytes apart fall into few memory channels, and
// workgroups in step would all ask the same ones (us, begun at 0 and turned: k
// 4096, n 4096, 16 experts, 24 rows 65 and 51, 200 rows 65, 47, 1000 rows 82,
// 71; k 8192, n 2048, 1000 rows 79, 72; but k 2048, n 7168, 1000 rows 54.6, 56.0).
__device__ __forceinline__ int first_turn(int32_t k, int64_t column_block, int group, int turns) {
  return k % 4096 != 0 ? 0 : static_cast<int>((column_block * 3 + group * int64_t(5)) % turns);
}

// Four consecutive columns of one row, as far as the row goes.
template <Out kOut>
__device__ __forceinline__ void store_columns(const GemmDeqArgs& a, int64_t row, int col, const float (&v)[4]) {
  const int64_t at = row * a.n + col;
  if (col + 4 <= a.n) {
    if constexpr (kOut == Out::kF32)
      *reinterpret_cast<f32x4_u*>(static_cast<float*>(a.out) + at) = f32x4{v[0], v[1], v[2], v[3]};
    else
      *reinterpret_cast<u32x2_u*>(static_cast<uint16_t*>(a.out) + at) =
          u32x2{pack2<kOut == Out::kFp16>(v[0], v[1]), pack2<kOut == Out::kFp16>(v[2], v[3])};
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (col + q < a.n) store_float<kOut>(a.out, at + q, round_f32(v[q]));
  }
}

// 16 bytes of consecutive columns of one row, as far as the row goes;
// non-temporally where the call says so.
template <Out kOut>
__device__ __forceinline__ void store_piece(const GemmDeqArgs& a, int64_t row, int col, const u32x4& bits) {
  constexpr int kSize = kOut == Out::kF32 ? 4 : 2, kCols = 16 / kSize;
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
      if constexpr (kOut == Out::kF32) static_cast<uint32_t*>(a.out)[at + q] = bits[q];
      else static_cast<uint16_t*>(a.out)[at + q] = static_cast<uint16_t>(bits[q / 2] >> (q % 2 * 16));
    }
  }
}

// ---- few rows for each expert -----------------------------------------------------

template <Out kOut, int kMI, int kNI, int kWaves, int kKC, int kSplit>
__global__ __launch_bounds__(kWave* kWaves* kSplit) void stream_kernel(GemmDeqArgs a, int64_t slots) {
  constexpr int kThreads = kWave * kWaves, kCols = 16 * kNI * kWaves;  // of one part
  constexpr int kRowPieces = kKC / 16;
  constexpr int kSteps = kKC / 64;
  constexpr int kCopies = kMI * 16 * kRowPieces / kThreads;  // pieces of a chunk's rows that a thread brings
  static_assert(kRowPieces % 16 == 0 && kCopies * kThreads == kMI * 16 * kRowPieces, "whole chunks");
  constexpr int kRowsBytes = kMI * 16 * kKC;
  __shared__ __attribute__((aligned(1024))) uint8_t rows0[kSplit * kRowsBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t rows1[kSplit * kRowsBytes];
  const int tid = threadIdx.x % kThreads, lane = tid % kWave, wave = uniform(tid / kWave);
  const int part = kSplit == 1 ? 0 : uniform(threadIdx.x / kThreads);
  uint8_t* const sa0 = rows0 + part * kRowsBytes;
  uint8_t* const sa1 = rows1 + part * kRowsBytes;
  // workgroups of one block of columns lie on one XCD, an expert's slots next to each other
  const int64_t x = blockIdx.x % 8, y = blockIdx.x / 8;
  const int64_t slot = y % slots, block = y / slots * 8 + x;
  if (block * kCols >= a.n) return;
  RowSlot rs;
  if (!find_row_slot<kMI * 16>(a.group_count, a.groups, a.rows, slot, lane, &rs)) return;

  const int col0 = static_cast<int>(block) * kCols + wave * 16 * kNI;
  const int piece = lane / 16 * 16;
  const int8_t* pb[kNI];
#pragma unroll
  for (int j = 0; j < kNI; ++j)
    pb[j] = a.w + (static_cast<int64_t>(rs.group) * a.n + min(col0 + j * 16 + lane % 16, a.n - 1)) * a.k;
  const int8_t* pa[kCopies];
  int ka[kCopies], la[kCopies];
#pragma unroll
  for (int q = 0; q < kCopies; ++q) {
    const int p = q * kThreads + tid, r = p / kRowPieces, c = p % kRowPieces;
    pa[q] = a.a + tile_row(rs.row0, rs.row_end, r) * a.a_stride;
    ka[q] = c * 16;
    la[q] = r * kKC + (c ^ (r % 16)) * 16;
  }
  float w[kNI][4], ts[kMI];
  const float* ws = a.weight_scale + static_cast<int64_t>(rs.group) * a.n;
#pragma unroll
  for (int j = 0; j < kNI; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) w[j][q] = ws[min(col0 + j * 16 + lane / 16 * 4 + q, a.n - 1)];
#pragma unroll
  for (int i = 0; i < kMI; ++i)
    ts[i] = *reinterpret_cast<const float*>(a.token_scale +
                                            tile_row(rs.row0, rs.row_end, i * 16 + lane % 16) * a.ts_stride);
  const int rounds = (a.k + kSplit * kKC - 1) / (kSplit * kKC);
  const int start = first_turn(a.k, block, rs.group, rounds);
  const auto turn = [&](int r) { return r + start < rounds ? r + start : r + start - rounds; };
  // Past k the rows count as zero, and whatever weights a valid address gives do no harm.
  auto load_a = [&](int round, i32x4 (&v)[kCopies]) {
    const int chunk = turn(round) * kSplit + part;
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const int at = chunk * kKC + ka[q];
      v[q] = *reinterpret_cast<const i32x4*>(pa[q] + (at < a.k ? at : 0));
      if (at >= a.k) v[q] = i32x4{0, 0, 0, 0};
    }
  };
  auto put_a = [&](uint8_t* buf, const i32x4 (&v)[kCopies]) {
#pragma unroll
    for (int q = 0; q < kCopies; ++q) *reinterpret_cast<i32x4*>(buf + la[q]) = v[q];
  };
  auto load_b = [&](int round, i32x4 (&v)[kSteps][kNI]) {
    const int chunk = turn(round) * kSplit + part;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int at = chunk * kKC + s * 64 + piece;
#pragma unroll
      for (int j = 0; j < kNI; ++j) v[s][j] = *reinterpret_cast<const i32x4*>(pb[j] + (at < a.k ? at : 0));
    }
  };
  i32x4 acc[kMI][kNI];
#pragma unroll
  for (int i = 0; i < kMI; ++i)
#pragma unroll
    for (int j = 0; j < kNI; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  auto multiply = [&](const uint8_t* buf, const i32x4 (&b)[kSteps][kNI]) {
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
      for (int i = 0; i < kMI; ++i) {
        const i32x4 f = *reinterpret_cast<const i32x4*>(buf + (i * 16 + lane % 16) * kKC +
                                                        ((s * 4 + lane / 16) ^ (lane % 16)) * 16);
#pragma unroll
        for (int j = 0; j < kNI; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[s][j], f, acc[i][j], 0, 0, 0);
      }
    }
  };

  i32x4 va0[kCopies], va1[kCopies], b0[kSteps][kNI], b1[kSteps][kNI];
  load_a(0, va0);
  load_b(0, b0);
  if (rounds > 1) {
    load_a(1, va1);
    load_b(1, b1);
  }
  put_a(sa0, va0);
  __syncthreads();
  // A buffer is written again only after the barrier that follows its readers.
  for (int c = 0;; c += 2) {
    multiply(sa0, b0);
    if (c + 1 >= rounds) break;
    if (c + 2 < rounds) {
      load_a(c + 2, va0);
      load_b(c + 2, b0);
    }
    put_a(sa1, va1);
    __syncthreads();
    multiply(sa1, b1);
    if (c + 2 >= rounds) break;
    if (c + 3 < rounds) {
      load_a(c + 3, va1);
      load_b(c + 3, b1);
    }
    put_a(sa0, va0);
    __syncthreads();
  }
  if constexpr (kSplit > 1) {  // the first part adds the others' sums
    static_assert((kSplit - 1) * kThreads * kMI * kNI * 16 <= kSplit * kRowsBytes, "the sums fit over the rows");
    i32x4* const sums = reinterpret_cast<i32x4*>(rows0);
    __syncthreads();
    if (part > 0) {
#pragma unroll
      for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int j = 0; j < kNI; ++j) sums[((part - 1) * kMI * kNI + i * kNI + j) * kThreads + tid] = acc[i][j];
    }
    __syncthreads();
    if (part > 0) return;
#pragma unroll
    for (int p = 1; p < kSplit; ++p)
#pragma unroll
      for (int i = 0; i < kMI; ++i)
#pragma unroll
        for (int j = 0; j < kNI; ++j) acc[i][j] += sums[((p - 1) * kMI * kNI + i * kNI + j) * kThreads + tid];
  }

#pragma unroll
  for (int j = 0; j < kNI; ++j) {
    const int col = col0 + j * 16 + lane / 16 * 4;
    if (col >= a.n) continue;
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
      const int r = i * 16 + lane % 16;
      if (tile_has_row(rs.row0, rs.row_end, r)) {
        float v[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = static_cast<float>(acc[i][j][q]) * w[j][q] * ts[i];
        store_columns<kOut>(a, rs.row0 + r, col, v);
      }
    }
  }
}

int64_t stream_blocks(int32_t rows, int32_t groups, int32_t n, int tile_m, int tile_n) {
  return row_slots(rows, groups, tile_m) * (((static_cast<int64_t>(n) + tile_n - 1) / tile_n + 7) / 8 * 8);
}

template <Out kOut, int kMI, int kNI, int kWaves, int kKC, int kSplit = 1>
hipError_t launch_stream(const GemmDeqArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(stream_blocks(a.rows, a.groups, a.n, kMI * 16, 16 * kNI * kWaves)));
  stream_kernel<kOut, kMI, kNI, kWaves, kKC, kSplit>
      <<<grid, dim3(kWave * kWaves * kSplit), 0, stream>>>(a, row_slots(a.rows, a.groups, kMI * 16));
  return hipGetLastError();
}

// ---- many rows for each expert -----------------------------------------------------

constexpr int kTileWaves = 8;
constexpr int kSK = 128;         // bytes of k per stage
constexpr int kGroupCols = 1024;  // columns of a group of column tiles

constexpr int vmcnt_wait(int n) { return 0x0f70 | (n & 15) | ((n >> 4) << 14); }
constexpr int kLgkmWait0 = 0xc07f;

// Position of a 16-byte piece in a stage row: piece p of row r sits at p ^
// swizzle(r).  The fragments read 16 rows at one piece, rows 16 i + (0 .. 15)
// of the rows and 32 p + {0-3, 8-11, 16-19, 24-27} (+ 4) of the weights; for
// both the 16 rows fall into all 16 groups of banks.
__device__ __forceinline__ int swizzle(int r) { return ((r >> 1) & 7) ^ (((r >> 4) & 1) << 1); }

template <Out kOut, int kTileM, int kTileN, int kWavesM, bool kTail>
__global__ __launch_bounds__(kWave* kTileWaves) void tile_kernel(GemmDeqArgs a) {
  constexpr int kWavesN = kTileWaves / kWavesM;
  constexpr int kWaveM = kTileM / kWavesM, kWaveN = kTileN / kWavesN;
  constexpr int kMI = kWaveM / 16, kNI = kWaveN / 16;
  constexpr int kRowsPerLoad = kWave / (kSK / 16);
  constexpr int kLoadsA = kTileM / kRowsPerLoad / kTileWaves, kLoadsB = kTileN / kRowsPerLoad / kTileWaves;
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
  const int64_t n_tiles = (a.n + kTileN - 1) / kTileN;
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
  const int col0 = static_cast<int>(col_tile) * kTileN;

  // Load q of this wave fills the stage rows from 8 (q 8 + wave); lane l
  // fetches the piece that belongs at position l % 8 of row l / 8, the same
  // piece for every q.
  const int piece = (lane % 8) ^ swizzle(kRowsPerLoad * wave + lane / 8);
  const int8_t* src_a[kLoadsA];
  const int8_t* src_b[kLoadsB];
#pragma unroll
  for (int q = 0; q < kLoadsA; ++q) {
    const int r = kRowsPerLoad * (q * kTileWaves + wave) + lane / 8;
    src_a[q] = a.a + tile_row(row0, row_end, r) * a.a_stride + piece * 16;
  }
#pragma unroll
  for (int q = 0; q < kLoadsB; ++q) {
    const int r = kRowsPerLoad * (q * kTileWaves + wave) + lane / 8;
    src_b[q] = a.w + (static_cast<int64_t>(rs.group) * a.n + min(col0 + r, a.n - 1)) * a.k + piece * 16;
  }
  // The scales before the loop where the registers allow it (2 % at 1000 rows).
  const int wm = wave / kWavesN, wn = wave % kWavesN;
  const int l16 = lane % 16;
  const int col_base = col0 + wn * kWaveN + 8 * (lane / 16);
  constexpr bool kEarlyScales = kMI * kNI <= 16;
  float ts[kMI], w[kNI / 2][8];
  const auto load_scales = [&]() {
    const float* ws = a.weight_scale + static_cast<int64_t>(rs.group) * a.n;
#pragma unroll
    for (int i = 0; i < kMI; ++i)
      ts[i] = *reinterpret_cast<const float*>(a.token_scale +
                                              tile_row(row0, row_end, wm * kWaveM + i * 16 + l16) * a.ts_stride);
#pragma unroll
    for (int p = 0; p < kNI / 2; ++p)
#pragma unroll
      for (int q = 0; q < 8; ++q) w[p][q] = ws[min(col_base + p * 32 + q, a.n - 1)];
  };
  if constexpr (kEarlyScales) load_scales();
  const int stages = (a.k + kSK - 1) / kSK;
  // Stages past the last one load it again, into slots that are not read; a
  // piece past k reads the row's first piece (its row fragments count as zero).
  // An expert's tiles in step, so that they share their rows and weights in L2;
  // the tile of 256 rows is not bound by its loads.  (A k with a tail begins at 0.)
  constexpr bool kTurned = kTileM < 256 && !kTail;
  const int start = kTurned ? first_turn(a.k, 0, rs.group, stages) : 0;
  const auto turn = [&](int s) { return !kTurned || s + start < stages ? s + start : s + start - stages; };
  auto stage_offset = [&](int s) {
    const int k0 = turn(min(s, stages - 1)) * kSK;
    if constexpr (kTail) return (k0 + piece * 16 < a.k) ? k0 : -piece * 16;
    return k0;
  };
  auto issue_a = [&](int s, uint8_t* buf) {
    const int off = stage_offset(s);
#pragma unroll
    for (int q = 0; q < kLoadsA; ++q) {
      const int8_t* src = src_a[q] + off;
      __builtin_amdgcn_global_load_lds(src, (MOE_LDS void*)(buf + (q * kTileWaves + wave) * kRowsPerLoad * kSK), 16, 0,
                                       0);
    }
  };
  auto issue_b = [&](int s, uint8_t* buf) {
    const int off = stage_offset(s);
#pragma unroll
    for (int q = 0; q < kLoadsB; ++q) {
      const int8_t* src = src_b[q] + off;
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
  i32x4 acc[kMI][kNI];
#pragma unroll
  for (int i = 0; i < kMI; ++i)
#pragma unroll
    for (int j = 0; j < kNI; ++j) acc[i][j] = i32x4{0, 0, 0, 0};

  auto barrier = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_s_barrier();
    __atomic_signal_fence(__ATOMIC_SEQ_CST);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](int S, int h, const uint8_t* ca, const uint8_t* cb, uint8_t* fill_a, uint8_t* fill_b) {
    if (h == 0) issue_a(S + 1, fill_a);  // into the slot A(S - 1) used
    else issue_b(S + 2, fill_b);         // into the slot B(S - 1) used
    const int p = 4 * h + lane / 16;
    i32x4 af[kMI], bf[kNI];
#pragma unroll
    for (int i = 0; i < kMI; ++i)
      af[i] = *reinterpret_cast<const i32x4*>(ca + frag_a + i * 16 * kSK + (p ^ swz_a ^ ((i & 1) << 1)) * 16);
#pragma unroll
    for (int j = 0; j < kNI; ++j)
      bf[j] = *reinterpret_cast<const i32x4*>(cb + frag_b + ((j >> 1) * 32 + (j & 1) * 4) * kSK +
                                              (p ^ swz_b ^ ((j & 1) << 1)) * 16);
    if constexpr (kTail) {
      const int keep = S * kSK + p * 16 < a.k ? -1 : 0;
#pragma unroll
      for (int i = 0; i < kMI; ++i) af[i] &= keep;
    }
    // this wave's loads of A(S + 1) and B(S + 1); those of B(S + 2) may still run
    if (h == 1) __builtin_amdgcn_s_waitcnt(vmcnt_wait(kLoadsB));
    __builtin_amdgcn_s_waitcnt(kLgkmWait0);
    barrier();
#pragma unroll
    for (int i = 0; i < kMI; ++i)
#pragma unroll
      for (int j = 0; j < kNI; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[j], af[i], acc[i][j], 0, 0, 0);
    barrier();
  };
  auto stage = [&](int S, const uint8_t* ca, const uint8_t* cb, uint8_t* fill_a, uint8_t* fill_b) {
    step(S, 0, ca, cb, fill_a, fill_b);
    step(S, 1, ca, cb, fill_a, fill_b);
  };
  issue_b(0, sb0);
  issue_a(0, sa0);
  issue_b(1, sb1);
  __builtin_amdgcn_s_waitcnt(vmcnt_wait(kLoadsB));
  barrier();
  const int grp = wave / 4;
  if (grp == 1) barrier();  // the second group runs half a step behind
  const int rounds = stages / 6;
  for (int r = 0; r < rounds; ++r) {
    stage(6 * r, sa0, sb0, sa1, sb2);
    stage(6 * r + 1, sa1, sb1, sa0, sb0);
    stage(6 * r + 2, sa0, sb2, sa1, sb1);
    stage(6 * r + 3, sa1, sb0, sa0, sb2);
    stage(6 * r + 4, sa0, sb1, sa1, sb0);
    stage(6 * r + 5, sa1, sb2, sa0, sb1);
  }
  {
    const int rest = stages - rounds * 6;
    if (rest > 0) stage(6 * rounds, sa0, sb0, sa1, sb2);
    if (rest > 1) stage(6 * rounds + 1, sa1, sb1, sa0, sb0);
    if (rest > 2) stage(6 * rounds + 2, sa0, sb2, sa1, sb1);
    if (rest > 3) stage(6 * rounds + 3, sa1, sb0, sa0, sb2);
    if (rest > 4) stage(6 * rounds + 4, sa0, sb1, sa1, sb0);
  }
  if (grp == 0) barrier();  // every wave passes the same number of barriers
  // no load may still be writing this workgroup's LDS
  __builtin_amdgcn_s_waitcnt(vmcnt_wait(0));

  if constexpr (!kEarlyScales) load_scales();
  // 16 rows of results at a time through LDS, so that a store's lanes lie along
  // rows (whole cache lines; stored from the products' layout, 64 bytes of each
  // of 16 rows, 32768 rows took 495 us instead of 469).  The weights' slots are
  // free once every wave's loads have landed and its reads are done.
  barrier();
  constexpr int kPieceCols = kOut == Out::kF32 ? 4 : 8;  // columns of a 16-byte piece
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
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = static_cast<float>(acc[i][2 * p + q / 4][q % 4]) * w[p][q] * ts[i];
      const int c = (p * 4 + lane / 16) * (8 / kPieceCols);
      if constexpr (kOut == Out::kF32) {
        *reinterpret_cast<f32x4*>(place(l16, c)) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(place(l16, c + 1)) = f32x4{v[4], v[5], v[6], v[7]};
      } else {
        constexpr bool kFp16 = kOut == Out::kFp16;
        *reinterpret_cast<u32x4*>(place(l16, c)) = u32x4{pack2<kFp16>(v[0], v[1]), pack2<kFp16>(v[2], v[3]),
                                                         pack2<kFp16>(v[4], v[5]), pack2<kFp16>(v[6], v[7])};
      }
    }
    wave_lds_sync();
#pragma unroll
    for (int t = 0; t < 16 * kRowPieces / kWave; ++t) {
      const int r = (t * kWave + lane) / kRowPieces, c = (t * kWave + lane) % kRowPieces;
      const u32x4 bits = *reinterpret_cast<const u32x4*>(place(r, c));
      const int tr = wm * kWaveM + i * 16 + r;
      if (tile_has_row(row0, row_end, tr)) store_piece<kOut>(a, row0 + tr, col0 + wn * kWaveN + c * kPieceCols, bits);
    }
    wave_lds_sync();
  }
}

int64_t tile_blocks(int32_t rows, int32_t groups, int32_t n, int tile_m, int tile_n) {
  return (row_slots(rows, groups, tile_m) * ((static_cast<int64_t>(n) + tile_n - 1) / tile_n) + 7) / 8 * 8;
}

template <Out kOut, int kTileM, int kTileN, int kWavesM>
hipError_t launch_tile(const GemmDeqArgs& a, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(tile_blocks(a.rows, a.groups, a.n, kTileM, kTileN))), block(kWave * kTileWaves);
  if (a.k % kSK != 0) tile_kernel<kOut, kTileM, kTileN, kWavesM, true><<<grid, block, 0, stream>>>(a);
  else tile_kernel<kOut, kTileM, kTileN, kWavesM, false><<<grid, block, 0, stream>>>(a);
  return hipGetLastError();
}

// One case for each tile of select::gemm_deq_kind.
template <Out kOut>
hipError_t launch_out(const GemmDeqArgs& a, hipStream_t stream) {
  const select::GemmDeqKind kind = select::gemm_deq_kind(a.rows, a.groups, a.n);
  const bool short_chunks = select::gemm_deq_short_chunks(kind, a.k);
  switch (kind) {
    case select::GemmDeqKind::kSplit16: return launch_stream<kOut, 1, 1, 1, 256, 4>(a, stream);
    case select::GemmDeqKind::kStream16:
      return short_chunks ? launch_stream<kOut, 1, 1, 4, 256>(a, stream)
                          : launch_stream<kOut, 1, 1, 2, 256, 2>(a, stream);
    case select::GemmDeqKind::kStream32:
      return short_chunks ? launch_stream<kOut, 2, 1, 4, 256>(a, stream) : launch_stream<kOut, 2, 1, 4, 512>(a, stream);
    case select::GemmDeqKind::kTile64: return launch_tile<kOut, 64, 128, 2>(a, stream);
    case select::GemmDeqKind::kTile128: return launch_tile<kOut, 128, 128, 2>(a, stream);
    case select::GemmDeqKind::kTile256: return launch_tile<kOut, 256, 256, 4>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

bool grouped_gemm_deq_fits(int32_t rows, int32_t groups, int32_t n) {
  constexpr int64_t kStreamBlocks = kMaxLaunchThreads / (4 * kWave);  // four waves, in one part of k or more
  constexpr int64_t kTileBlocks = kMaxLaunchThreads / (kTileWaves * kWave);
  switch (select::gemm_deq_kind(rows, groups, n)) {
    case select::GemmDeqKind::kSplit16: return stream_blocks(rows, groups, n, 16, 16) <= kStreamBlocks;
    case select::GemmDeqKind::kStream16:  // (64 columns for a short k)
      return stream_blocks(rows, groups, n, 16, 32) <= kStreamBlocks;
    case select::GemmDeqKind::kStream32: return stream_blocks(rows, groups, n, 32, 64) <= kStreamBlocks;
    case select::GemmDeqKind::kTile64: return tile_blocks(rows, groups, n, 64, 128) <= kTileBlocks;
    case select::GemmDeqKind::kTile128: return tile_blocks(rows, groups, n, 128, 128) <= kTileBlocks;
    case select::GemmDeqKind::kTile256: return tile_blocks(rows, groups, n, 256, 256) <= kTileBlocks;
  }
  return false;
}

hipError_t launch_grouped_gemm_deq(GemmDeqArgs a, Out out_type, hipStream_t stream) {
  if (a.rows == 0) return hipSuccess;
  if (!grouped_gemm_deq_fits(a.rows, a.groups, a.n)) return hipErrorInvalidValue;
  a.nt = select::gemm_deq_nt(a.rows, a.groups, a.k, a.n, out_type == Out::kF32 ? 4 : 2);
  switch (out_type) {
    case Out::kBf16: return launch_out<Out::kBf16>(a, stream);
    case Out::kFp16: return launch_out<Out::kFp16>(a, stream);
    case Out::kF32: return launch_out<Out::kF32>(a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace moe
