// A running sum over a workgroup, shared by the kernels of a step over the paged cache.
#pragma once

#include "pbg_device.hpp"

namespace pbg {

// Sum of v over the threads before this one, and over all threads (W whole waves).
template <int W, typename V>
__device__ __forceinline__ V block_scan(V v, V* waves, V& total) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  V s = v;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const V o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  __syncthreads();  // the last use of waves
  if (lane == kWave - 1) waves[wave] = s;
  __syncthreads();
  V before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < wave) before += waves[w];
    total += waves[w];
  }
  return before + s - v;
}

}  // namespace pbg
