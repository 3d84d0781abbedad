// Scans and searches of the mapping launches (workgroups of kMapThreads).
#pragma once

#include <cstdint>

#include "tcl_internal.hpp"

namespace tcl {

constexpr int kMapThreads = 1024;

// Inclusive scan over a wave by lane moves: 1, 2, 4 and 8 lanes inside each
// row of 16, then the last lane of rows 0 and 2 into the row behind, then the
// last lane of row 1 into rows 2 and 3.  ROWS false: inside rows only.
template <bool ROWS>
__device__ inline int lane_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  if constexpr (ROWS) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  }
  return v;
}

// Exclusive scans of N numbers a thread over the workgroup: v becomes the sum
// before the thread, total the workgroup's.
template <int N>
__device__ inline void block_scan(int (&v)[N], int (&total)[N], int (*lds)[kMapThreads / 64]) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  constexpr int W = kMapThreads / 64;
  static_assert(W == 16, "the waves' sums fill a row of lanes");
  int inc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) inc[i] = lane_scan<true>(v[i]);
  __syncthreads();
  if (lane == 63) {
#pragma unroll
    for (int i = 0; i < N; ++i) lds[i][w] = inc[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    // the waves' sums, scanned by every wave
    const int x = lds[i][lane & (W - 1)], y = lane_scan<false>(x);
    total[i] = __builtin_amdgcn_readlane(y, W - 1);
    v[i] = inc[i] - v[i] + __builtin_amdgcn_readlane(y - x, w);
  }
}

__device__ inline int upper(const int32_t *ptr, int n, int x) {
  // the last i in [0, n) with ptr[i] <= x
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (ptr[m] <= x)
      lo = m;
    else
      hi = m;
  }
  return lo;
}

}  // namespace tcl
