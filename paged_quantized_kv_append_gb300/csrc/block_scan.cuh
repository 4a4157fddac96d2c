// Sums over a block's threads and a search in what they leave: the block tables and
// the shared prefixes' plan lay requests (groups) end to end with them.
#pragma once

#include <stdint.h>

namespace pqkv {

// Exclusive sums over the block's threads of two per-thread values; the totals come back
// in ta and tb.
template <int kThreads, class A, class B>
__device__ __forceinline__ void block_scan2(A& a, B& b, A& ta, B& tb) {
  __shared__ A wa[kThreads / 32];
  __shared__ B wb[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  A ia = a;
  B ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const A ua = __shfl_up_sync(0xffffffffu, ia, o);
    const B ub = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) {
      ia += ua;
      ib += ub;
    }
  }
  __syncthreads();                       // the sums of a scan before this one are read
  if (lane == 31) {
    wa[warp] = ia;
    wb[warp] = ib;
  }
  __syncthreads();
  A ba = 0;
  B bb = 0;
  ta = 0;
  tb = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w == warp) {
      ba = ta;
      bb = tb;
    }
    ta += wa[w];
    tb += wb[w];
  }
  a = ba + ia - a;
  b = bb + ib - b;
}

// The last of n ascending entries that is at most x (the first one is).
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

}  // namespace pqkv
