// Device helpers of the attention kernels: matrix products of 32 x 32 tiles and
// what goes with their layout. A product's lane holds 16 rows of ONE column
// (lane % 32): element i is row 8 (i / 4) + 4 (lane / 32) + i % 4.
#pragma once

#include "seq_device.h"

namespace emb {

typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef _Float16 hf8 __attribute__((ext_vector_type(8)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s4v lds_s4v;

constexpr float kNegInf = -__builtin_inff();

template <int DT>
__device__ __forceinline__ f16v mfma(s8v a, s8v b, f16v c) {
  if constexpr (DT == EMB_BF16)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(hf8, a), __builtin_bit_cast(hf8, b), c, 0, 0, 0);
}

template <int DT>
__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const fl2 f = {x, y};
  if constexpr (DT == EMB_BF16) return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf2));
  else return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, hf2));
}

// A row's two lanes (l and l + 32) joined.
__device__ __forceinline__ void halves(float x, float* lo, float* hi) {
  typedef unsigned u2v __attribute__((ext_vector_type(2)));
  const u2v r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  *lo = __uint_as_float(r.x);
  *hi = __uint_as_float(r.y);
}
__device__ __forceinline__ float both_halves_max(float x) {
  float lo, hi;
  halves(x, &lo, &hi);
  return fmaxf(lo, hi);
}
__device__ __forceinline__ float both_halves_sum(float x) {
  float lo, hi;
  halves(x, &lo, &hi);
  return lo + hi;
}

// The last i in [0, n) with f(i) <= x, f non-decreasing, by one wave: 64
// places at a time.
template <class F>
__device__ __forceinline__ int wave_find(int n, int x, F f) {
  const int lane = threadIdx.x & 63;
  int lo = 0, len = n;
  while (len > 1) {
    const int step = (len + 63) >> 6;
    const int i = lo + lane * step;
    const bool le = lane * step < len && f(i) <= x;
    const uint64_t mask = __ballot(le);
    const int k = mask ? 63 - __clzll(mask) : 0;
    const int at = k * step;
    len = min(step, len - at);
    lo += at;
  }
  return lo;
}

template <int N>
__device__ __forceinline__ float top_of(const f16v (&s)[N]) {
  float top = s[0][0];
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = n == 0; i < 16; ++i) top = fmaxf(top, s[n][i]);
  return top;
}

// Clears the scores of a tile's slots at and beyond `seen` (the lane's own limit).
__device__ __forceinline__ void mask_tile(f16v& s, int slot0, int seen) {
  const int h4 = 4 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (slot0 + 8 * (i / 4) + h4 + i % 4 >= seen) s[i] = kNegInf;
}

}  // namespace emb
