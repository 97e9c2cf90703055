// What the kernels of the block tables share: the CTA's shape, its prefix sums, and the
// segment of a table row that one warp moves.
#pragma once

#include "common.cuh"

namespace dflash {

namespace pages {
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSegment = 128;            // pages that a warp moves at once
}  // namespace pages

// Exclusive prefix of one value per thread over the block, and the total.
__device__ __forceinline__ long long block_prefix(long long x, long long* total) {
  __shared__ long long s_w[pages::kWarps];
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  long long in = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, in, o);
    if (l >= o) in += y;
  }
  __syncthreads();   // the array may still be read from the call before
  if (l == 31) s_w[w] = in;
  __syncthreads();
  long long base = 0, all = 0;
#pragma unroll
  for (int i = 0; i < pages::kWarps; ++i) {
    const long long v = s_w[i];
    base += i < w ? v : 0;
    all += v;
  }
  *total = all;
  return base + in - x;
}

}  // namespace dflash
