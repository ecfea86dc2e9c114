// Prefix sums of a workgroup of 1024 threads.
#pragma once

#include <hip/hip_runtime.h>

#include "tq_common.h"

namespace tq {

constexpr int kScanThreads = 1024;

// Exclusive prefix sum over the workgroup and its total.
template <class T>
__device__ __forceinline__ T scan_block(T v, T* red, T& total) {
  const int t = threadIdx.x, lane = t & 63, w = t >> 6;
  T inc = v;
#pragma unroll
  for (int off = 1; off < kWave; off <<= 1) {
    const T o = __shfl_up(inc, off, kWave);
    inc += lane >= off ? o : T(0);
  }
  __syncthreads();  // red of the previous call has been read
  if (lane == 63) red[w] = inc;
  __syncthreads();
  T before = inc - v;
  total = 0;
#pragma unroll
  for (int i = 0; i < kScanThreads / kWave; ++i) {
    const T r = red[i];
    before += i < w ? r : T(0);
    total += r;
  }
  return before;
}

}  // namespace tq
