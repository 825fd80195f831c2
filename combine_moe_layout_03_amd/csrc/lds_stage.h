// Stages of k in LDS, as the matrix products' tiles fill, wait for and read them.
#pragma once

#include <hip/hip_runtime.h>

namespace moe {

#define MOE_LDS __attribute__((address_space(3)))  // what an LDS-destination load writes to

// s_waitcnt with vmcnt(n) (expcnt and lgkmcnt left at their maxima).
constexpr int vmcnt_wait(int n) { return 0x0f70 | (n & 15) | ((n >> 4) << 14); }
// s_waitcnt with lgkmcnt(0) (vmcnt and expcnt left at their maxima).
constexpr int kLgkmWait0 = 0xc07f;

// The plain s_barrier, with nothing moved across it.  (The fence of
// __syncthreads would wait for every load in flight.)
__device__ __forceinline__ void tile_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_sched_barrier(0);
}

// Position of a 16-byte piece in a stage row of 128 bytes: piece p of row r sits
// at p ^ swizzle(r).  The fragments read 16 rows at one piece, rows 16 i + (0 ..
// 15) of the rows and 32 p + {0-3, 8-11, 16-19, 24-27} (+ 4) of the weights; for
// both the 16 rows fall into all 16 groups of banks.
__device__ __forceinline__ int swizzle(int r) { return ((r >> 1) & 7) ^ (((r >> 4) & 1) << 1); }

}  // namespace moe
