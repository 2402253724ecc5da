// Device helpers of the sequence operators' and the history layer's kernels.
#pragma once

#include "emb_device.h"
#include "seq_internal.h"

namespace emb {

template <int DT>
struct Elem {
  using T = uint16_t;
};
template <>
struct Elem<EMB_F32> {
  using T = float;
};

template <int DT>
__device__ __forceinline__ float ld1(const void* p, long long i) {
  if constexpr (DT == EMB_F32) return reinterpret_cast<const float*>(p)[i];
  else return half_to_f32<DT>(reinterpret_cast<const uint16_t*>(p)[i]);
}
template <int DT>
__device__ __forceinline__ void st1(void* p, long long i, float x) {
  if constexpr (DT == EMB_F32) reinterpret_cast<float*>(p)[i] = x;
  else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)f32_to_half<DT>(x);
}

// Conversions of the vector paths: the hardware's, to nearest even with
// subnormals kept (the default mode of these kernels).
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef _Float16 hf2 __attribute__((ext_vector_type(2)));
typedef float fl2 __attribute__((ext_vector_type(2)));

template <int DT>
__device__ __forceinline__ void widen(const u4 v, float* out) {
  if constexpr (DT == EMB_F16) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const hf2 h = __builtin_bit_cast(hf2, w[i]);
      out[2 * i] = (float)h.x;
      out[2 * i + 1] = (float)h.y;
    }
  } else {
    widen16<DT>(v, out);
  }
}

template <int DT>
__device__ __forceinline__ u4 narrow(const float* in) {
  if constexpr (DT == EMB_F32) {
    return u4{__float_as_uint(in[0]), __float_as_uint(in[1]), __float_as_uint(in[2]), __float_as_uint(in[3])};
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const fl2 f = {in[2 * i], in[2 * i + 1]};
      if constexpr (DT == EMB_BF16) w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf2));
      else w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, hf2));
    }
    return u4{w[0], w[1], w[2], w[3]};
  }
}

// Sum over the lanes of a group of G neighbours (a power of two, at most 32):
// lane exchanges inside rows of 16 are operand modifiers, not LDS traffic.
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float near_sum(float x, int G) {
  if (G > 1) x += dpp<0xB1>(x);   // swap neighbours
  if (G > 2) x += dpp<0x4E>(x);   // swap pairs
  if (G > 4) x += dpp<0x141>(x);  // mirror 8 lanes: quads are uniform by now
  if (G > 8) x += dpp<0x140>(x);  // mirror 16 lanes
  if (G > 16) x += __shfl_xor(x, 16, 64);
  return x;
}

__device__ __forceinline__ int div_by(const FastDiv d, int n) {
  return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift);
}

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
