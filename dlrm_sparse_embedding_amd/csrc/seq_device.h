// Device helpers of the sequence operators' kernels (k_rotary.hip, k_prefix.hip).
#pragma once

#include "emb_device.h"
#include "seq_internal.h"

namespace emb {

// Whether offsets [n + 1] break their contract (first 0, never decreasing, last
// `end`) between a at i and b at i + 1.
__device__ __forceinline__ bool breaks_offsets(int a, int b, long long i, int n, int end) {
  return a > b || (i == 0 && a != 0) || (i == n - 1 && b != end);
}

// Raises the flag for them: each neighbouring pair is looked at by one thread of
// the grid of 256-thread blocks.
__device__ __forceinline__ void report_offsets(const int* offsets, int n, int end, int* error) {
  if (!error) return;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256)
    if (breaks_offsets(offsets[i], offsets[i + 1], i, n, end)) atomicOr(error, kKvBadOffsets);
}

}  // namespace emb
