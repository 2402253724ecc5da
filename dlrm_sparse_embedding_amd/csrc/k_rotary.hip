// Rotary positions, the per-head norm of queries and keys with the rotation in
// the same pass, its gradient, and the append of keys and values to a paged
// cache with both applied on the way.
//
// Mathematics. A head x of dim elements, pairs (a_i, b_i) among its first rot:
//   forward   y = R(x r w),  r = (mean x^2 + eps)^(-1/2),  R = turn by pos f_i, times mag
//   gradient  u = R^T dy,  n = x r,  dx = r (u w - n mean(u w n)),  dw = sum u n
// All of it is one pass over the heads: bound by memory. Angles are integers:
// pair i's frequency is a 64-bit fraction of a turn, so position * frequency
// modulo 2^64 loses nothing but the frequency's rounding times the position
// (2^-31 of a turn at 2^32); sine and cosine come from the Taylor series on an eighth of a turn to either side of a quadrant's
// middle (terms to x^9 and x^10, truncation below 5e-9).
//
// Layout. A lane owns one "unit": 2 V elements (V = 16 bytes' worth) that hold
// V whole pairs, as two 16-byte accesses: V elements at p and V at p + rot/2
// (half layout) or p + V (interleaved), so one set of sines serves a unit in
// either layout. The lanes of a head are a power of two of neighbours, so the
// norm's sum is a few lane exchanges. Operands that 16-byte accesses do not
// fit go through the element-wise kernels below.
//
// Measured (a large copy reaches 5.4 TB/s read and written): rotation of 16384 x
// 32 x 64 fp32 58 us (4.6 TB/s), norm of 16384 x 40 x 128 bf16 62 us (5.4), its
// gradient for 12289 tokens 97 us (3.9; the vector units are 43% busy, neither
// more loads in flight nor more blocks change it), append of 20011 x 8 x 128
// bf16 with norm 39 us (4.2; rows scattered over pages). Small calls are bound by
// the launch: 3 to 5 us on the device, 7 to 9 through the binding.
#include <algorithm>

#include "seq_device.h"

namespace emb {

namespace {

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

// Sine and cosine of pos * turn / 2^64 turns. The phase's upper 32 bits are
// kept (2^-32 of a turn); what is left after the nearest quarter is at most an
// eighth of a turn, up to 2^29 units, which fp32 rounds by up to 16: 2^-28 of a
// turn, less than half a step of fp32 at 1.
__device__ __forceinline__ void sincos_turn(uint64_t turn, long long pos, float mag, float* c, float* s) {
  const uint32_t ph = (uint32_t)((turn * (uint64_t)pos) >> 32);
  const uint32_t quad = (ph + 0x20000000u) >> 30;
  const float x = (float)(int)(ph - (quad << 30)) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float z = x * x;
  const float sn = x + x * z * (-1.f / 6 + z * (1.f / 120 + z * (-1.f / 5040 + z * (1.f / 362880))));
  const float cs = 1.f + z * (-0.5f + z * (1.f / 24 + z * (-1.f / 720 + z * (1.f / 40320 + z * (-1.f / 3628800)))));
  const float a = (quad & 1) ? sn : cs;  // |cos|
  const float b = (quad & 1) ? cs : sn;  // |sin|
  *c = ((quad + 1) & 2) ? -mag * a : mag * a;
  *s = (quad & 2) ? -mag * b : mag * b;
}

__device__ __forceinline__ long long position(const void* p, int itype, long long t) {
  return itype == EMB_I64 ? reinterpret_cast<const long long*>(p)[t] : (long long)reinterpret_cast<const int*>(p)[t];
}

// Sum over the lanes of a group of G neighbours (G a power of two).
__device__ __forceinline__ float group_sum(float x, int G) {
  for (int d = 1; d < G; d <<= 1) x += __shfl_xor(x, d, 64);
  return x;
}

// ---- element by element ------------------------------------------------------
// One wave for each head; lane l owns pairs l, l + 64, .. and the elements
// behind the rotation. Right for every dim, rot, stride and alignment.

// Pair i's two elements.
__device__ __forceinline__ void pair_at(const RotTable& rot, int i, int* ea, int* eb) {
  if (rot.layout == EMB_ROT_HALF) {
    *ea = i;
    *eb = i + rot.rot / 2;
  } else {
    *ea = 2 * i;
    *eb = 2 * i + 1;
  }
}

// y = rotate(x [* r * w]) for one head, by one wave.
template <int DT>
__device__ void head_any(const void* x, long long xi, void* y, long long yi, int dim, const RotTable& rot,
                         long long pos, float sign, bool norm, const float* w, float eps) {
  const int lane = threadIdx.x & 63;
  float r = 1.f;
  if (norm) {
    float ss = 0.f;
    for (int e = lane; e < dim; e += 64) {
      const float v = ld1<DT>(x, xi + e);
      ss += v * v;
    }
    r = 1.f / sqrtf(group_sum(ss, 64) / (float)dim + eps);
  }
  for (int i = lane; i < rot.rot / 2; i += 64) {
    int ea, eb;
    pair_at(rot, i, &ea, &eb);
    float c, s;
    sincos_turn(rot.turn[i], pos, rot.mag, &c, &s);
    s *= sign;
    const float a = ld1<DT>(x, xi + ea) * r * (w ? w[ea] : 1.f);
    const float b = ld1<DT>(x, xi + eb) * r * (w ? w[eb] : 1.f);
    st1<DT>(y, yi + ea, a * c - b * s);
    st1<DT>(y, yi + eb, a * s + b * c);
  }
  for (int e = rot.rot + lane; e < dim; e += 64) {
    if (norm) {
      st1<DT>(y, yi + e, ld1<DT>(x, xi + e) * r * (w ? w[e] : 1.f));
    } else {
      using T = typename Elem<DT>::T;
      reinterpret_cast<T*>(y)[yi + e] = reinterpret_cast<const T*>(x)[xi + e];
    }
  }
}

template <int DT>
__global__ __launch_bounds__(256) void k_norm_rotary_any(NormRotaryArgs a, RotTable rot) {
  const int H = a.q.n + a.k.n;
  for (long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); item < a.tokens * H;
       item += (long long)gridDim.x * 4) {
    const long long t = item / H;
    const int h = (int)(item - t * H);
    const bool isq = h < a.q.n;
    const Heads& in = isq ? a.q : a.k;
    const Heads& out = isq ? a.qo : a.ko;
    const int hh = isq ? h : h - a.q.n;
    head_any<DT>(in.p, t * in.ts + hh * in.hs, const_cast<void*>(out.p), t * out.ts + hh * out.hs, a.dim, rot,
                 position(a.positions, a.itype, t), a.inverse ? -1.f : 1.f, a.norm, isq ? a.wq : a.wk, a.eps);
  }
}

// Gradient, element by element. Each wave takes heads in turn; it sums the
// weights' gradients of its heads in LDS, the block's waves are joined at the
// end in their order.
template <int DT>
__global__ __launch_bounds__(256) void k_norm_rotary_back_any(NormRotaryBackArgs a, RotTable rot) {
  extern __shared__ float s_dw[];  // [4][2][dim]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int dim = a.dim;
  for (int i = threadIdx.x; i < 8 * dim; i += 256) s_dw[i] = 0.f;
  __syncthreads();
  const int H = a.q.n + a.k.n;
  for (long long item = (long long)blockIdx.x * 4 + wave; item < a.tokens * H; item += (long long)gridDim.x * 4) {
    const long long t = item / H;
    const int h = (int)(item - t * H);
    const bool isq = h < a.q.n;
    const int hh = isq ? h : h - a.q.n;
    const Heads& in = isq ? a.q : a.k;
    const Heads& dy = isq ? a.dyq : a.dyk;
    const Heads& dx = isq ? a.dq : a.dk;
    const float* w = isq ? a.wq : a.wk;
    float* dw = s_dw + (wave * 2 + (isq ? 0 : 1)) * dim;
    const long long xi = t * in.ts + hh * in.hs, yi = t * dy.ts + hh * dy.hs, oi = t * dx.ts + hh * dx.hs;
    const long long pos = position(a.positions, a.itype, t);
    float ss = 0.f;
    for (int e = lane; e < dim; e += 64) {
      const float v = ld1<DT>(in.p, xi + e);
      ss += v * v;
    }
    const float r = 1.f / sqrtf(group_sum(ss, 64) / (float)dim + a.eps);
    // twice over the head: first the mean of u w n, then the gradient
    float dot = 0.f;
    for (int pass = 0; pass < 2; ++pass) {
      const float mean = pass ? group_sum(dot, 64) / (float)dim : 0.f;
      auto one = [&](int e, float u) {
        const float n = ld1<DT>(in.p, xi + e) * r;
        const float g = u * (w ? w[e] : 1.f);
        if (pass == 0) {
          dot += g * n;
        } else {
          dw[e] += u * n;  // element e is this lane's alone
          st1<DT>(const_cast<void*>(dx.p), oi + e, r * (g - n * mean));
        }
      };
      for (int i = lane; i < rot.rot / 2; i += 64) {
        int ea, eb;
        pair_at(rot, i, &ea, &eb);
        float c, s;
        sincos_turn(rot.turn[i], pos, rot.mag, &c, &s);
        const float da = ld1<DT>(dy.p, yi + ea), db = ld1<DT>(dy.p, yi + eb);
        const float ua = da * c + db * s, ub = db * c - da * s;
        one(ea, ua);
        one(eb, ub);
      }
      for (int e = rot.rot + lane; e < dim; e += 64) one(e, ld1<DT>(dy.p, yi + e));
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * dim; i += 256) {
    float s = 0.f;
    for (int w = 0; w < 4; ++w) s += s_dw[w * 2 * dim + i];
    a.part[(long long)blockIdx.x * 2 * dim + i] = s;
  }
}

// Weights' gradients from the blocks' partial sums, in 64 bits: 4 columns for
// each block, a row of them for each thread, so that (with up to 1280 rows) all
// loads are under way at once.
__global__ __launch_bounds__(256) void k_norm_dw(const float* __restrict__ part, int blocks, int dim,
                                                 float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ double s[4][256];
  const int col = blockIdx.x * 4;
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  for (int b0 = threadIdx.x; b0 < blocks; b0 += 5 * 256) {
    float x[5][4];
#pragma unroll
    for (int i = 0; i < 5; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int b = b0 + 256 * i;
        x[i][c] = b < blocks && col + c < 2 * dim ? part[(long long)b * 2 * dim + col + c] : 0.f;
      }
#pragma unroll
    for (int i = 0; i < 5; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[c] += (double)x[i][c];
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) s[c][threadIdx.x] = acc[c];
  __syncthreads();
  // a wave for each column
  const int c = threadIdx.x >> 6, lane = threadIdx.x & 63;
  double sum = s[c][lane] + s[c][lane + 64] + s[c][lane + 128] + s[c][lane + 192];
  for (int d = 32; d >= 1; d >>= 1) sum += __shfl_down(sum, d, 64);
  if (lane == 0 && col + c < 2 * dim) {
    float* out = col + c < dim ? dwq : dwk;
    if (out) out[col + c < dim ? col + c : col + c - dim] = (float)sum;
  }
}

// ---- 16-byte units ---------------------------------------------------------------

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

template <int DT>
constexpr int kV = DT == EMB_F32 ? 4 : 8;  // elements of 16 bytes

// A lane's unit of 2 V elements.
template <int DT, int LAYOUT>
struct Unit {
  static constexpr int V = kV<DT>;
  int e0, e1;     // its two runs of V elements
  bool turns;     // it holds pairs
  float c[V], s[V];

  __device__ __forceinline__ void place(int u, const RotTable& rot) {
    turns = 2 * V * u < rot.rot;
    e0 = 2 * V * u;
    e1 = e0 + V;
    if (LAYOUT == EMB_ROT_HALF && turns) {
      e0 = V * u;
      e1 = rot.rot / 2 + V * u;
    }
  }
  __device__ __forceinline__ void angles(int u, const RotTable& rot, long long pos, float sign) {
    if (!turns) return;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      sincos_turn(rot.turn[V * u + j], pos, rot.mag, &c[j], &s[j]);
      s[j] *= sign;
    }
  }
  // x: the unit's elements, run 0 then run 1
  __device__ __forceinline__ void turn(float* x) const {
    if (!turns) return;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int ia = LAYOUT == EMB_ROT_HALF ? j : 2 * j, ib = LAYOUT == EMB_ROT_HALF ? V + j : 2 * j + 1;
      const float a = x[ia], b = x[ib];
      x[ia] = a * c[j] - b * s[j];
      x[ib] = a * s[j] + b * c[j];
    }
  }
};

// 16 bytes at element i. Every element is read once, so reads pass the L2 by;
// writes do (PAST) where a store instruction fills whole lines. Together with
// neighbouring heads in a wave's accesses: an append of 20011 tokens 48 -> 42 us,
// norm of 16384 x 40 heads 76 -> 68, its gradient 105 -> 99. Parts of lines that pass the L2 by are written several times (rotation
// of half of each 192-byte head 27 -> 45 us).
template <int DT>
__device__ __forceinline__ u4 get16(const void* p, long long i) {
  return __builtin_nontemporal_load(reinterpret_cast<const u4*>(reinterpret_cast<const typename Elem<DT>::T*>(p) + i));
}
template <int DT, bool PAST = false>
__device__ __forceinline__ void put16(const void* p, long long i, u4 x) {
  u4* at = reinterpret_cast<u4*>(reinterpret_cast<typename Elem<DT>::T*>(const_cast<void*>(p)) + i);
  if (PAST) __builtin_nontemporal_store(x, at);
  else *at = x;
}
template <int DT, bool PAST = false>
__device__ __forceinline__ void put16(const void* p, long long i, const float* x) {
  put16<DT, PAST>(p, i, narrow<DT>(x));
}

// The unit's part of a weight (ones where it is null).
template <int V>
__device__ __forceinline__ void load_w(const float* w, int e0, int e1, float* out) {
#pragma unroll
  for (int j = 0; j < 2 * V; ++j) out[j] = 1.f;
  if (!w) return;
#pragma unroll
  for (int j = 0; j < V; j += 4) {
    load4<EMB_F32>(w + e0 + j, out + j);
    load4<EMB_F32>(w + e1 + j, out + V + j);
  }
}

// The lanes of a call: groups of G lanes (units of them busy), one group for
// HPT heads of one token, so that one set of angles serves them all; queries
// and keys are never in one group, so a group has one weight. A group's heads
// lie gq (gk) apart: a wave's accesses then cover neighbouring heads.
struct VecShape {
  int G, units;
  int gq, gk;      // head groups of the queries (values, in the append: of the keys) and of the keys (values)
  FastDiv by_g;    // by gq + gk
  long long items; // tokens * (gq + gk) < 2^31
};

template <int DT, int LAYOUT, int NORM, int HPT, bool PAST>
__global__ __launch_bounds__(256, 4) void k_norm_rotary_vec(NormRotaryArgs a, VecShape sh, RotTable rot) {
  constexpr int V = kV<DT>;
  const int u = threadIdx.x & (sh.G - 1);
  const int per = 256 / sh.G;
  const bool busy = u < sh.units;
  Unit<DT, LAYOUT> un;
  un.place(u, rot);
  for (long long item = (long long)blockIdx.x * per + threadIdx.x / sh.G; item < sh.items;
       item += (long long)gridDim.x * per) {
    const int t = (int)(((uint64_t)(uint32_t)item * sh.by_g.mul) >> sh.by_g.shift);
    const int g = (int)item - t * (int)sh.by_g.d;
    const bool isq = g < sh.gq;
    const Heads& in = isq ? a.q : a.k;
    const Heads& out = isq ? a.qo : a.ko;
    const int h0 = isq ? g : g - sh.gq, hs = isq ? sh.gq : sh.gk;  // heads h0, h0 + hs, ..
    u4 lo[HPT], hi[HPT];
    if (busy) {
#pragma unroll
      for (int i = 0; i < HPT; ++i) {
        const int h = min(h0 + i * hs, in.n - 1);
        lo[i] = get16<DT>(in.p, t * in.ts + h * in.hs + un.e0);
        hi[i] = get16<DT>(in.p, t * in.ts + h * in.hs + un.e1);
      }
      un.angles(u, rot, position(a.positions, a.itype, t), a.inverse ? -1.f : 1.f);
    }
    float w[2 * V];
    if (NORM) {
      if (busy) load_w<V>(isq ? a.wq : a.wk, un.e0, un.e1, w);
    }
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
      float x[2 * V];
      if (busy) {
        widen<DT>(lo[i], x);
        widen<DT>(hi[i], x + V);
      }
      if (NORM) {
        float ss = 0.f;
        if (busy) {
#pragma unroll
          for (int j = 0; j < 2 * V; ++j) ss += x[j] * x[j];
        }
        const float r = 1.f / sqrtf(near_sum(ss, sh.G) / (float)a.dim + a.eps);
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) x[j] *= r * w[j];
      }
      if (busy && h0 + i * hs < in.n) {
        const long long yi = t * out.ts + (h0 + i * hs) * out.hs;
        if (!NORM && !un.turns) {  // a copy, whatever the bits
          put16<DT>(out.p, yi + un.e0, lo[i]);
          put16<DT>(out.p, yi + un.e1, hi[i]);
        } else {
          un.turn(x);
          put16<DT, PAST>(out.p, yi + un.e0, x);
          put16<DT, PAST>(out.p, yi + un.e1, x + V);
        }
      }
    }
  }
}

// Gradient. The grid's groups are a multiple of the head groups, so a group
// stays on one head group and sums one weight's gradient in its registers over
// all its tokens; the block's groups are joined through LDS in their order.
constexpr int kBackHeads = 4;

template <int DT, int LAYOUT, bool PAST>
__global__ __launch_bounds__(256, 3) void k_norm_rotary_back_vec(NormRotaryBackArgs a, VecShape sh, RotTable rot) {
  constexpr int V = kV<DT>;
  __shared__ float s_dw[256 * 2 * V];
  const int u = threadIdx.x & (sh.G - 1);
  const int per = 256 / sh.G;
  const bool busy = u < sh.units;
  const int HG = sh.gq + sh.gk;
  Unit<DT, LAYOUT> un;
  un.place(u, rot);
  const long long first = (long long)blockIdx.x * per + threadIdx.x / sh.G;
  const int g = (int)(first % HG);
  const bool isq = g < sh.gq;
  const Heads& in = isq ? a.q : a.k;
  const Heads& dyh = isq ? a.dyq : a.dyk;
  const Heads& dxh = isq ? a.dq : a.dk;
  const int h0 = isq ? g : g - sh.gq, hs = isq ? sh.gq : sh.gk;  // heads h0, h0 + hs, ..
  float w[2 * V], dw[2 * V];
#pragma unroll
  for (int j = 0; j < 2 * V; ++j) dw[j] = 0.f;
  if (busy) load_w<V>(isq ? a.wq : a.wk, un.e0, un.e1, w);
  for (long long t = first / HG; t < a.tokens; t += (long long)gridDim.x * per / HG) {
    if (busy) un.angles(u, rot, position(a.positions, a.itype, t), -1.f);
#pragma unroll
    for (int i = 0; i < kBackHeads; ++i) {
      const int h = h0 + i * hs;
      if (h >= in.n) break;  // the same for all lanes of the group
      float x[2 * V], d[2 * V], ss = 0.f, dot = 0.f;
      if (busy) {
        const long long xi = t * in.ts + h * in.hs, yi = t * dyh.ts + h * dyh.hs;
        widen<DT>(get16<DT>(in.p, xi + un.e0), x);
        widen<DT>(get16<DT>(in.p, xi + un.e1), x + V);
        widen<DT>(get16<DT>(dyh.p, yi + un.e0), d);
        widen<DT>(get16<DT>(dyh.p, yi + un.e1), d + V);
        un.turn(d);
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) {
          ss += x[j] * x[j];
          dot += d[j] * w[j] * x[j];
        }
      }
      const float r = 1.f / sqrtf(near_sum(ss, sh.G) / (float)a.dim + a.eps);
      const float mean = near_sum(dot, sh.G) * r / (float)a.dim;
      if (busy) {
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) {
          const float n = x[j] * r;
          dw[j] += d[j] * n;
          d[j] = r * (d[j] * w[j] - n * mean);
        }
        const long long oi = t * dxh.ts + h * dxh.hs;
        put16<DT, PAST>(dxh.p, oi + un.e0, d);
        put16<DT, PAST>(dxh.p, oi + un.e1, d + V);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < 2 * V; ++j) s_dw[threadIdx.x * 2 * V + j] = busy ? dw[j] : 0.f;
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.dim; i += 256) {
    const bool wantq = i < a.dim;
    const int e = wantq ? i : i - a.dim;
    // unit and place of element e
    int uu = e / (2 * V), j = e % (2 * V);
    if (LAYOUT == EMB_ROT_HALF && e < rot.rot) {
      const int half = rot.rot / 2, ee = e < half ? e : e - half;
      uu = ee / V;
      j = ee % V + (e < half ? 0 : V);
    }
    float sum = 0.f;
    for (int q = 0; q < per; ++q) {
      const int gg = (int)(((long long)blockIdx.x * per + q) % HG);
      if ((gg < sh.gq) == wantq) sum += s_dw[(q * sh.G + uu) * 2 * V + j];
    }
    a.part[(long long)blockIdx.x * 2 * a.dim + i] = sum;
  }
}

// ---- the append -----------------------------------------------------------------

// The sequence of token t: the last b with offsets[b] <= t.
__device__ __forceinline__ int seq_of(const int* offsets, int seqs, int t) {
  int lo = 0, hi = seqs;  // offsets[lo] <= t < offsets[hi] by contract
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (offsets[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int div_by(const FastDiv d, int n) {
  return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift);
}

// Page and slot in it of token t; false where it has none. *slot is the slot
// in the sequence.
__device__ __forceinline__ bool place(const AppendArgs& a, int t, int* page, int* in_page, int* slot) {
  int b = t, first = t, n = 1;
  if (a.offsets) {
    b = seq_of(a.offsets, a.seqs, t);
    first = a.offsets[b];
    const int next = a.offsets[b + 1];
    if (first < 0 || t < first || t >= next || next > a.tokens) {  // offsets that do not cover the token, or more
      if (a.kv.error) atomicOr(a.kv.error, kKvBadOffsets);
      return false;
    }
    n = next - first;
  }
  const long long s = (long long)a.lens[b] - n + (t - first);
  if (s < 0 || s >= (long long)a.width * a.kv.page) {
    if (a.kv.error) atomicOr(a.kv.error, kKvBadPage);
    return false;
  }
  const int col = div_by(a.kv.by_page, (int)s);
  const int p = a.table[(long long)b * a.width + col];
  if (p < 0 || p >= a.kv.pages) {
    if (a.kv.error) atomicOr(a.kv.error, kKvBadPage);
    return false;
  }
  *page = p;
  *in_page = (int)s - col * a.kv.page;
  *slot = (int)s;
  return true;
}

template <int DT>
__global__ __launch_bounds__(256) void k_append_any(AppendArgs a, RotTable rot) {
  const int H = 2 * a.kv.heads;
  const KvView& kv = a.kv;
  if (a.offsets) report_offsets(a.offsets, a.seqs, (int)a.tokens, kv.error);
  for (long long item = (long long)blockIdx.x * 4 + (threadIdx.x >> 6); item < a.tokens * H;
       item += (long long)gridDim.x * 4) {
    const long long t = item / H;
    const int h = (int)(item - t * H);
    int page, in_page, slot;
    if (!place(a, (int)t, &page, &in_page, &slot)) continue;
    if (h < kv.heads) {
      const long long pos = a.positions ? position(a.positions, a.itype, t) : (long long)slot;
      head_any<DT>(a.k.p, t * a.k.ts + h * a.k.hs, kv.k, page * kv.kps + in_page * kv.kss + h * kv.khs, kv.dim, rot,
                   pos, 1.f, a.norm, a.wk, a.eps);
    } else {
      using T = typename Elem<DT>::T;
      const int hv = h - kv.heads;
      const T* src = reinterpret_cast<const T*>(a.v.p) + t * a.v.ts + hv * a.v.hs;
      T* dst = reinterpret_cast<T*>(kv.v) + (page * kv.vps + in_page * kv.vss + hv * kv.vhs);
      for (int e = threadIdx.x & 63; e < kv.dim; e += 64) dst[e] = src[e];
    }
  }
}

template <int DT, int LAYOUT, int HPT>
__global__ __launch_bounds__(256, 4) void k_append_vec(AppendArgs a, VecShape sh, RotTable rot) {
  constexpr int V = kV<DT>;
  const KvView& kv = a.kv;
  const int u = threadIdx.x & (sh.G - 1);
  const int per = 256 / sh.G;
  const bool busy = u < sh.units;
  Unit<DT, LAYOUT> un;
  un.place(u, rot);
  if (a.offsets) report_offsets(a.offsets, a.seqs, (int)a.tokens, kv.error);
  for (long long item = (long long)blockIdx.x * per + threadIdx.x / sh.G; item < sh.items;
       item += (long long)gridDim.x * per) {
    const int t = (int)(((uint64_t)(uint32_t)item * sh.by_g.mul) >> sh.by_g.shift);
    const int g = (int)item - t * (int)sh.by_g.d;
    const bool isk = g < sh.gq;
    const Heads& in = isk ? a.k : a.v;
    const int h0 = isk ? g : g - sh.gq, step = isk ? sh.gq : sh.gk;  // heads h0, h0 + step, ..
    u4 lo[HPT], hi[HPT];
    if (busy) {
#pragma unroll
      for (int i = 0; i < HPT; ++i) {
        const int h = min(h0 + i * step, in.n - 1);
        lo[i] = get16<DT>(in.p, t * in.ts + h * in.hs + un.e0);
        hi[i] = get16<DT>(in.p, t * in.ts + h * in.hs + un.e1);
      }
    }
    int page, in_page, slot;
    if (!place(a, t, &page, &in_page, &slot)) continue;  // the same for all lanes of the group
    char* out = isk ? kv.k : kv.v;
    const long long row = isk ? page * kv.kps + in_page * kv.kss : page * kv.vps + in_page * kv.vss;
    const long long hs = isk ? kv.khs : kv.vhs;
    float w[2 * V];
    if (isk && busy) {
      un.angles(u, rot, a.positions ? position(a.positions, a.itype, t) : (long long)slot, 1.f);
      if (a.norm) load_w<V>(a.wk, un.e0, un.e1, w);
    }
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
      const bool store = busy && h0 + i * step < in.n;
      const long long yi = row + (h0 + i * step) * hs;
      if (!isk || (!a.norm && !un.turns)) {
        if (store) {
          put16<DT>(out, yi + un.e0, lo[i]);
          put16<DT>(out, yi + un.e1, hi[i]);
        }
        if (!isk || !a.norm) continue;
      }
      float x[2 * V];
      if (busy) {
        widen<DT>(lo[i], x);
        widen<DT>(hi[i], x + V);
      }
      if (a.norm) {
        float ss = 0.f;
        if (busy) {
#pragma unroll
          for (int j = 0; j < 2 * V; ++j) ss += x[j] * x[j];
        }
        const float r = 1.f / sqrtf(near_sum(ss, sh.G) / (float)kv.dim + a.eps);
#pragma unroll
        for (int j = 0; j < 2 * V; ++j) x[j] *= r * w[j];
      }
      if (store) {
        un.turn(x);
        put16<DT>(out, yi + un.e0, x);
        put16<DT>(out, yi + un.e1, x + V);
      }
    }
  }
}

// Whether 16-byte units fit an operand.
bool fits(const Heads& h, int dtype) {
  const int V = dtype == EMB_F32 ? 4 : 8;
  return h.n == 0 || (reinterpret_cast<uintptr_t>(h.p) % 16 == 0 && h.ts % V == 0 && h.hs % V == 0);
}

// Units of the calls over dim elements with this rotation; G = 0 where they do not fit.
VecShape vec_shape(int dtype, int dim, const RotTable& rot, long long tokens, int nq, int nk, int hpt) {
  VecShape sh{};
  const int V2 = dtype == EMB_F32 ? 8 : 16;
  sh.gq = (nq + hpt - 1) / hpt;
  sh.gk = (nk + hpt - 1) / hpt;
  sh.items = tokens * (sh.gq + sh.gk);
  if (dim % V2 != 0 || rot.rot % V2 != 0 || dim / V2 > 32 || sh.items >= (1ll << 31)) return sh;
  sh.units = dim / V2;
  sh.G = 1;
  while (sh.G < sh.units) sh.G *= 2;
  sh.by_g = fast_div((uint32_t)(sh.gq + sh.gk));
  return sh;
}

unsigned vec_grid(const VecShape& sh) {
  const int per = 256 / sh.G;
  return (unsigned)std::min<long long>((sh.items + per - 1) / per, 1 << 20);
}

// Whether a store instruction's 16-byte pieces of one run fill whole lines of an operand.
bool whole_lines(const Heads& h, int dtype, int dim, const RotTable& rot) {
  const int es = dtype == EMB_F32 ? 4 : 2;
  return h.n == 0 || (rot.layout == EMB_ROT_HALF && rot.rot == dim && dim / 2 * es % 128 == 0 &&
                      reinterpret_cast<uintptr_t>(h.p) % 128 == 0 && h.ts * es % 128 == 0 && h.hs * es % 128 == 0);
}

// Heads for each group of lanes. Four share their angles and keep 128 bytes a
// lane in flight; with little work one head each spreads it over the chip.
int heads_per_group(long long tokens, int heads, int units) {
  return tokens * heads * units >= (1ll << 20) ? 4 : 1;
}

template <int DT, int LAYOUT, int NORM>
void launch_vec(const NormRotaryArgs& a, const VecShape& sh, int hpt, const RotTable& rot, hipStream_t st) {
  // little work stays in the L2 for who reads it next
  const bool past = hpt == 4 && whole_lines(a.qo, DT, a.dim, rot) && whole_lines(a.ko, DT, a.dim, rot);
  if (past) k_norm_rotary_vec<DT, EMB_ROT_HALF, NORM, 4, true><<<vec_grid(sh), 256, 0, st>>>(a, sh, rot);
  else if (hpt == 4) k_norm_rotary_vec<DT, LAYOUT, NORM, 4, false><<<vec_grid(sh), 256, 0, st>>>(a, sh, rot);
  else k_norm_rotary_vec<DT, LAYOUT, NORM, 1, false><<<vec_grid(sh), 256, 0, st>>>(a, sh, rot);
}

template <int DT>
void launch_vec_t(const NormRotaryArgs& a, const VecShape& sh, int hpt, const RotTable& rot, hipStream_t st) {
  if (rot.layout == EMB_ROT_HALF) {
    if (a.norm) launch_vec<DT, EMB_ROT_HALF, 1>(a, sh, hpt, rot, st);
    else launch_vec<DT, EMB_ROT_HALF, 0>(a, sh, hpt, rot, st);
  } else {
    if (a.norm) launch_vec<DT, EMB_ROT_INTERLEAVED, 1>(a, sh, hpt, rot, st);
    else launch_vec<DT, EMB_ROT_INTERLEAVED, 0>(a, sh, hpt, rot, st);
  }
}

template <int DT>
void launch_back_vec(const NormRotaryBackArgs& a, int blocks, const VecShape& sh, const RotTable& rot, hipStream_t st) {
  const bool past = whole_lines(a.dq, DT, a.dim, rot) && whole_lines(a.dk, DT, a.dim, rot);
  if (past) k_norm_rotary_back_vec<DT, EMB_ROT_HALF, true><<<blocks, 256, 0, st>>>(a, sh, rot);
  else if (rot.layout == EMB_ROT_HALF) k_norm_rotary_back_vec<DT, EMB_ROT_HALF, false><<<blocks, 256, 0, st>>>(a, sh, rot);
  else k_norm_rotary_back_vec<DT, EMB_ROT_INTERLEAVED, false><<<blocks, 256, 0, st>>>(a, sh, rot);
}

template <int DT, int LAYOUT>
void launch_append_vec(const AppendArgs& a, const VecShape& sh, int hpt, const RotTable& rot, hipStream_t st) {
  if (hpt == 4) k_append_vec<DT, LAYOUT, 4><<<vec_grid(sh), 256, 0, st>>>(a, sh, rot);
  else k_append_vec<DT, LAYOUT, 1><<<vec_grid(sh), 256, 0, st>>>(a, sh, rot);
}

template <int DT>
void launch_append_vec_t(const AppendArgs& a, const VecShape& sh, int hpt, const RotTable& rot, hipStream_t st) {
  if (rot.layout == EMB_ROT_HALF) launch_append_vec<DT, EMB_ROT_HALF>(a, sh, hpt, rot, st);
  else launch_append_vec<DT, EMB_ROT_INTERLEAVED>(a, sh, hpt, rot, st);
}

}  // namespace

hipError_t launch_norm_rotary(const NormRotaryArgs& a, const RotTable& rot, hipStream_t st) {
  if (fits(a.q, a.dtype) && fits(a.qo, a.dtype) && fits(a.k, a.dtype) && fits(a.ko, a.dtype)) {
    const int hpt = heads_per_group(a.tokens, a.q.n + a.k.n, a.dim / (a.dtype == EMB_F32 ? 8 : 16));
    const VecShape sh = vec_shape(a.dtype, a.dim, rot, a.tokens, a.q.n, a.k.n, hpt);
    if (sh.G > 0) {
      if (a.dtype == EMB_F32) launch_vec_t<EMB_F32>(a, sh, hpt, rot, st);
      else if (a.dtype == EMB_BF16) launch_vec_t<EMB_BF16>(a, sh, hpt, rot, st);
      else launch_vec_t<EMB_F16>(a, sh, hpt, rot, st);
      return hipGetLastError();
    }
  }
  const long long items = a.tokens * (a.q.n + a.k.n);
  const unsigned grid = (unsigned)std::min<long long>((items + 3) / 4, 1 << 20);
  if (a.dtype == EMB_F32) k_norm_rotary_any<EMB_F32><<<grid, 256, 0, st>>>(a, rot);
  else if (a.dtype == EMB_BF16) k_norm_rotary_any<EMB_BF16><<<grid, 256, 0, st>>>(a, rot);
  else k_norm_rotary_any<EMB_F16><<<grid, 256, 0, st>>>(a, rot);
  return hipGetLastError();
}

hipError_t launch_norm_rotary_back(const NormRotaryBackArgs& a, const RotTable& rot, hipStream_t st) {
  const int blocks = norm_rotary_back_blocks(a.tokens, a.q.n, a.k.n, a.dim);
  const bool fit = fits(a.q, a.dtype) && fits(a.dyq, a.dtype) && fits(a.dq, a.dtype) && fits(a.k, a.dtype) &&
                   fits(a.dyk, a.dtype) && fits(a.dk, a.dtype);
  const VecShape sh = vec_shape(a.dtype, a.dim, rot, a.tokens, a.q.n, a.k.n, kBackHeads);
  if (blocks > 0 && fit && sh.G > 0) {
    if (a.dtype == EMB_F32) launch_back_vec<EMB_F32>(a, blocks, sh, rot, st);
    else if (a.dtype == EMB_BF16) launch_back_vec<EMB_BF16>(a, blocks, sh, rot, st);
    else launch_back_vec<EMB_F16>(a, blocks, sh, rot, st);
    if (hipError_t e = hipGetLastError()) return e;
  } else if (blocks > 0) {
    const size_t lds = 8 * sizeof(float) * a.dim;
    if (a.dtype == EMB_F32) k_norm_rotary_back_any<EMB_F32><<<blocks, 256, lds, st>>>(a, rot);
    else if (a.dtype == EMB_BF16) k_norm_rotary_back_any<EMB_BF16><<<blocks, 256, lds, st>>>(a, rot);
    else k_norm_rotary_back_any<EMB_F16><<<blocks, 256, lds, st>>>(a, rot);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (a.dwq || a.dwk) k_norm_dw<<<(2 * a.dim + 3) / 4, 256, 0, st>>>(a.part, blocks, a.dim, a.dwq, a.dwk);
  return hipGetLastError();
}

hipError_t launch_kv_append(const AppendArgs& a, const RotTable& rot, hipStream_t st) {
  const KvView& c = a.kv;
  const Heads ck{c.k, c.kss, c.khs, c.heads}, cv{c.v, c.vss, c.vhs, c.heads};
  const int V = c.dtype == EMB_F32 ? 4 : 8;
  if (fits(a.k, c.dtype) && fits(a.v, c.dtype) && fits(ck, c.dtype) && fits(cv, c.dtype) && c.kps % V == 0 &&
      c.vps % V == 0) {
    const int hpt = heads_per_group(a.tokens, 2 * c.heads, c.dim / (2 * V));
    const VecShape sh = vec_shape(c.dtype, c.dim, rot, a.tokens, c.heads, c.heads, hpt);
    if (sh.G > 0) {
      if (c.dtype == EMB_F32) launch_append_vec_t<EMB_F32>(a, sh, hpt, rot, st);
      else if (c.dtype == EMB_BF16) launch_append_vec_t<EMB_BF16>(a, sh, hpt, rot, st);
      else launch_append_vec_t<EMB_F16>(a, sh, hpt, rot, st);
      return hipGetLastError();
    }
  }
  const long long items = a.tokens * 2 * a.kv.heads;
  const unsigned grid = (unsigned)std::min<long long>((items + 3) / 4, 1 << 20);
  if (a.kv.dtype == EMB_F32) k_append_any<EMB_F32><<<grid, 256, 0, st>>>(a, rot);
  else if (a.kv.dtype == EMB_BF16) k_append_any<EMB_BF16><<<grid, 256, 0, st>>>(a, rot);
  else k_append_any<EMB_F16><<<grid, 256, 0, st>>>(a, rot);
  return hipGetLastError();
}

}  // namespace emb
