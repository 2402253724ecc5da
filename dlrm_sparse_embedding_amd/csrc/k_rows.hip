// Layer norm of rows, its gradient, and dropout with a residual sum.
//
// Mathematics. For a row x of n elements, m = mean x, r = (mean (x - m)^2 +
// eps)^(-1/2), h = (x - m) r:
//   forward   y = h w + b
//   gradient  g = dy w,  dx = r (g - mean g - h mean(g h)),  dw = sum_rows dy h,
//             db = sum_rows dy
// One pass over the rows, which stay in registers between the mean and the
// variance; bound by memory. The weights' gradients are summed in fp32 along
// the rows of a group of lanes, in fp64 over the blocks, always in one order.
//
// Layout. A row belongs to a group of G lanes (a power of two, at most a wave)
// or, beyond 1024 columns, to a block; lane u holds the columns E (k G + u) ..
// + E - 1, k < K: each access of the group is one run of 16 bytes a lane. Rows
// that such accesses do not fit have E = 1.
#include <algorithm>

#include "seq_device.h"

namespace emb {

namespace {

typedef unsigned long long u64;

// E neighbouring elements from element i on, read and written once: past the L2.
template <int DT, int E>
__device__ __forceinline__ void get_unit(const void* p, long long i, float* out) {
  using T = typename Elem<DT>::T;
  const T* at = reinterpret_cast<const T*>(p) + i;
  if constexpr (E == 1) {
    out[0] = ld1<DT>(p, i);
  } else if constexpr (E * sizeof(T) == 16) {
    widen<DT>(__builtin_nontemporal_load(reinterpret_cast<const u4*>(at)), out);
  } else {
    static_assert(E * sizeof(T) == 8, "8 or 16 bytes");
    const u2 v = __builtin_nontemporal_load(reinterpret_cast<const u2*>(at));
    float f[8];
    widen<DT>(u4{v.x, v.y, 0, 0}, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = f[j];
  }
}
template <int DT, int E>
__device__ __forceinline__ void put_unit(const void* p, long long i, const float* in) {
  using T = typename Elem<DT>::T;
  T* at = reinterpret_cast<T*>(const_cast<void*>(p)) + i;
  if constexpr (E == 1) {
    st1<DT>(const_cast<void*>(p), i, in[0]);
  } else if constexpr (E * sizeof(T) == 16) {
    __builtin_nontemporal_store(narrow<DT>(in), reinterpret_cast<u4*>(at));
  } else {
    const float f[8] = {in[0], in[1], in[2], in[3]};
    const u4 v = narrow<DT>(f);
    __builtin_nontemporal_store(u2{v.x, v.y}, reinterpret_cast<u2*>(at));
  }
}
template <int E>
__device__ __forceinline__ void get_weight(const float* w, int i, float none, float* out) {
#pragma unroll
  for (int j = 0; j < E; ++j) out[j] = w ? w[i + j] : none;
}

// The lanes of a row.
template <int E, int K, bool BIG>
struct Place {
  int u, width;          // this lane, and how many there are
  long long row, step;   // the group's first row, and from one to the next
  __device__ __forceinline__ explicit Place(int G) {
    u = BIG ? threadIdx.x : threadIdx.x & (G - 1);
    width = BIG ? blockDim.x : G;
    const int per = BIG ? 1 : 256 / G;
    row = (long long)blockIdx.x * per + (BIG ? 0 : threadIdx.x / G);
    step = (long long)gridDim.x * per;
  }
  __device__ __forceinline__ int col(int k) const { return E * (k * width + u); }
};

// Sum over the row's lanes; `turn` alternates between a block's uses of it.
template <bool BIG>
__device__ __forceinline__ float row_sum(float x, int G, int turn, float (*s)[16]) {
  if constexpr (!BIG) {
    x = near_sum(x, min(G, 32));
    return G == 64 ? x + __shfl_xor(x, 32, 64) : x;
  } else {
    x = near_sum(x, 32);
    x += __shfl_xor(x, 32, 64);
    if ((threadIdx.x & 63) == 0) s[turn][threadIdx.x >> 6] = x;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < (int)(blockDim.x >> 6); ++i) t += s[turn][i];
    return t;
  }
}

// Mean and reciprocal deviation; x becomes the differences from the mean.
template <int E, int K, bool BIG>
__device__ __forceinline__ float center(const Place<E, K, BIG>& at, float (&x)[K * E], int dim, float eps, int G,
                                        float (*s)[16]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < K * E; ++i) sum += x[i];
  const float mean = row_sum<BIG>(sum, G, 0, s) / (float)dim;
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (at.col(k) < dim) {
#pragma unroll
      for (int j = 0; j < E; ++j) {
        x[k * E + j] -= mean;
        ss += x[k * E + j] * x[k * E + j];
      }
    }
  return 1.f / sqrtf(row_sum<BIG>(ss, G, 1, s) / (float)dim + eps);
}

template <int XT, int YT, int E, int K, bool BIG>
__global__ __launch_bounds__(BIG ? 1024 : 256) void k_layer_norm(LayerNormArgs a, int G) {
  __shared__ float s[2][16];
  const Place<E, K, BIG> at(G);
  float w[K * E], b[K * E];
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (at.col(k) < a.dim) {
      get_weight<E>(a.w, at.col(k), 1.f, w + k * E);
      get_weight<E>(a.b, at.col(k), 0.f, b + k * E);
    }
  for (long long row = at.row; row < a.rows; row += at.step) {
    float x[K * E] = {};
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at.col(k) < a.dim) get_unit<XT, E>(a.x.p, row * a.x.stride + at.col(k), x + k * E);
    const float r = center(at, x, a.dim, a.eps, G, s);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at.col(k) < a.dim) {
#pragma unroll
        for (int j = 0; j < E; ++j) x[k * E + j] = x[k * E + j] * r * w[k * E + j] + b[k * E + j];
        put_unit<YT, E>(a.y.p, row * a.y.stride + at.col(k), x + k * E);
      }
  }
}

template <int XT, int YT, int E, int K, bool BIG>
__global__ __launch_bounds__(BIG ? 1024 : 256) void k_layer_norm_back(LayerNormBackArgs a, int G) {
  __shared__ float s[2][16];
  __shared__ float s2[2][16];
  __shared__ float s_part[BIG ? 1 : 4 * 2 * 1024];
  const Place<E, K, BIG> at(G);
  float w[K * E], dw[K * E] = {}, db[K * E] = {};
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (at.col(k) < a.dim) get_weight<E>(a.w, at.col(k), 1.f, w + k * E);
  for (long long row = at.row; row < a.rows; row += at.step) {
    float x[K * E] = {}, dy[K * E] = {};
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at.col(k) < a.dim) {
        get_unit<XT, E>(a.x.p, row * a.x.stride + at.col(k), x + k * E);
        get_unit<YT, E>(a.dy.p, row * a.dy.stride + at.col(k), dy + k * E);
      }
    const float r = center(at, x, a.dim, a.eps, G, s);
    float sg = 0.f, sgh = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at.col(k) < a.dim) {
#pragma unroll
        for (int j = k * E; j < k * E + E; ++j) {
          x[j] *= r;  // h
          dw[j] += dy[j] * x[j];
          db[j] += dy[j];
          dy[j] *= w[j];  // g
          sg += dy[j];
          sgh += dy[j] * x[j];
        }
      }
    const float mg = row_sum<BIG>(sg, G, 0, s2) / (float)a.dim;
    const float mgh = row_sum<BIG>(sgh, G, 1, s2) / (float)a.dim;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at.col(k) < a.dim) {
#pragma unroll
        for (int j = k * E; j < k * E + E; ++j) x[j] = r * (dy[j] - mg - x[j] * mgh);
        put_unit<XT, E>(a.dx.p, row * a.dx.stride + at.col(k), x + k * E);
      }
  }
  if (!a.dw && !a.db) return;
  float* part = a.part + (long long)blockIdx.x * 2 * a.dim;
  if constexpr (BIG) {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at.col(k) < a.dim)
#pragma unroll
        for (int j = 0; j < E; ++j) {
          part[at.col(k) + j] = dw[k * E + j];
          part[a.dim + at.col(k) + j] = db[k * E + j];
        }
  } else {
    // the wave's groups, then the block's waves
    for (int d = G; d < 64; d <<= 1)
#pragma unroll
      for (int j = 0; j < K * E; ++j) {
        dw[j] += __shfl_xor(dw[j], d, 64);
        db[j] += __shfl_xor(db[j], d, 64);
      }
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) < G) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (at.col(k) < a.dim)
#pragma unroll
          for (int j = 0; j < E; ++j) {
            s_part[(wave * 2) * 1024 + at.col(k) + j] = dw[k * E + j];
            s_part[(wave * 2 + 1) * 1024 + at.col(k) + j] = db[k * E + j];
          }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.dim; i += 256) {
      const int half = i >= a.dim, c = i - half * a.dim;
      float t = 0.f;
#pragma unroll
      for (int v = 0; v < 4; ++v) t += s_part[(v * 2 + half) * 1024 + c];
      part[i] = t;
    }
  }
}

// Weights' gradients from the blocks' partial sums, in 64 bits: 32 columns for a
// block (whole lines), 32 rows of them at a time, 8 under way.
__global__ __launch_bounds__(1024) void k_layer_norm_dw(const float* __restrict__ part, int blocks, int dim,
                                                        float* __restrict__ dw, float* __restrict__ db) {
  __shared__ double s[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  double acc = 0.0;
  if (col < 2 * dim) {
    for (int b0 = slice; b0 < blocks; b0 += 8 * 32) {
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = b0 + 32 * i < blocks ? part[(long long)(b0 + 32 * i) * 2 * dim + col] : 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc += (double)x[i];
    }
  }
  s[slice][threadIdx.x & 31] = acc;
  __syncthreads();
  if (slice == 0 && col < 2 * dim) {
    double t = 0.0;
    for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
    if (col < dim) {
      if (dw) dw[col] = (float)t;
    } else if (db) {
      db[col - dim] = (float)t;
    }
  }
}

bool fits(const Rows2D& r, int E) {
  const int bytes = E * esize(r.dtype);
  return aligned(r.p, (size_t)bytes) && r.stride % E == 0;
}

// How a call's rows are laid out on lanes: E elements a unit (1 where an operand
// does not take wide accesses), 16 elements a lane at most. Small rows have one
// unit a lane.
struct Shape {
  int E, K, G, threads;  // G = 0: a block for each row
};
Shape shape_of(int dim, bool wide, bool any_f32) {
  Shape s{};
  s.E = wide ? (any_f32 ? 4 : 8) : 1;
  const int kmax = 16 / s.E, units = (dim + s.E - 1) / s.E;
  if (dim > 1024) {
    s.K = kmax;
    s.threads = dim <= 4096 ? 256 : 1024;
    return s;
  }
  s.threads = 256;
  s.K = units <= 8 ? 1 : kmax;
  s.G = 1;
  while (s.G * s.K < units) s.G *= 2;
  return s;
}

template <int XT, int YT, bool BACK, typename A>
hipError_t launch_norm(const A& a, bool wide, int cap, hipStream_t st, int* blocks) {
  constexpr int EV = XT == EMB_F32 || YT == EMB_F32 ? 4 : 8;
  const Shape s = shape_of(a.dim, wide, EV == 4);
  const int per = s.G ? 256 / s.G : 1;
  *blocks = (int)std::min<long long>((a.rows + per - 1) / per, cap);
  auto run = [&](auto kernel) { kernel<<<*blocks, s.threads, 0, st>>>(a, s.G); };
#define EMB_NORM(E, K, BIG)                                        \
  do {                                                             \
    if constexpr (BACK) run(k_layer_norm_back<XT, YT, E, K, BIG>); \
    else run(k_layer_norm<XT, YT, E, K, BIG>);                     \
  } while (0)
  if (s.E == 1) {
    if (s.G == 0) EMB_NORM(1, 16, true);
    else if (s.K == 1) EMB_NORM(1, 1, false);
    else EMB_NORM(1, 16, false);
  } else {
    if (s.G == 0) EMB_NORM(EV, 16 / EV, true);
    else if (s.K == 1) EMB_NORM(EV, 1, false);
    else EMB_NORM(EV, 16 / EV, false);
  }
#undef EMB_NORM
  return hipGetLastError();
}

template <bool BACK, typename A>
hipError_t launch_norm_types(const A& a, int xt, int yt, bool wide, int cap, hipStream_t st, int* blocks) {
  if (xt == EMB_BF16) return launch_norm<EMB_BF16, EMB_BF16, BACK>(a, wide, cap, st, blocks);
  if (xt == EMB_F16) return launch_norm<EMB_F16, EMB_F16, BACK>(a, wide, cap, st, blocks);
  if (yt == EMB_F32) return launch_norm<EMB_F32, EMB_F32, BACK>(a, wide, cap, st, blocks);
  if (yt == EMB_BF16) return launch_norm<EMB_F32, EMB_BF16, BACK>(a, wide, cap, st, blocks);
  return launch_norm<EMB_F32, EMB_F16, BACK>(a, wide, cap, st, blocks);
}

// ---- dropout -----------------------------------------------------------------

// Philox4x32-10: ten rounds of two 32 x 32 -> 64 bit products.
__device__ __forceinline__ void philox(uint32_t (&c)[4], uint64_t seed) {
  uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const u64 a = (u64)c[0] * 0xD2511F53u, b = (u64)c[2] * 0xCD9E8D57u;
    const uint32_t n0 = (uint32_t)(b >> 32) ^ c[1] ^ k0, n2 = (uint32_t)(a >> 32) ^ c[3] ^ k1;
    c[1] = (uint32_t)b;
    c[3] = (uint32_t)a;
    c[0] = n0;
    c[2] = n2;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// Which of the 8 elements of unit u of a row are kept, a bit each. Their upper
// 16 random bits decide but where they equal the threshold's (one in 65536):
// then the wave draws again, for the lower 16.
__device__ __forceinline__ uint32_t kept_bits(uint32_t u, uint32_t row, u64 step, u64 seed, u64 threshold) {
  const uint32_t c2 = (uint32_t)step, c3 = (uint32_t)(step >> 32) & 0x7fffffffu;
  const uint32_t top = (uint32_t)(threshold >> 16), low = (uint32_t)threshold & 0xffffu;
  uint32_t c[4] = {u, row, c2, c3};
  philox(c, seed);
  uint32_t keep = 0, tie = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t h = i & 1 ? c[i / 2] >> 16 : c[i / 2] & 0xffffu;
    keep |= (h > top ? 1u : 0u) << i;
    tie |= (h == top ? 1u : 0u) << i;
  }
  if (tie) {
    uint32_t d[4] = {u, row, c2, c3 | 0x80000000u};
    philox(d, seed);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t h = i & 1 ? d[i / 2] >> 16 : d[i / 2] & 0xffffu;
      if (h >= low) keep |= tie & (1u << i);
    }
  }
  return keep;
}

// Units row0 * units .. of n: 16-byte accesses, a unit of 8 elements a lane.
template <int DT>
__device__ __forceinline__ void get8(const void* p, long long i, float* x) {
  if constexpr (DT == EMB_F32) {
    get_unit<DT, 4>(p, i, x);
    get_unit<DT, 4>(p, i + 4, x + 4);
  } else {
    get_unit<DT, 8>(p, i, x);
  }
}

template <int DT, bool WIDE>
__global__ __launch_bounds__(256) void k_dropout(DropoutArgs a, FastDiv by_units, uint32_t row0, int n) {
  const u64 step = a.step ? (u64)*a.step : 0;
  const int lane = threadIdx.x & 63;
  // whole waves stay in the loop: lanes trade masks
  for (long long i0 = (long long)blockIdx.x * 256 + (threadIdx.x & ~63); i0 < n; i0 += (long long)gridDim.x * 256) {
    const bool on = i0 + lane < n;
    const int i = (int)min(i0 + lane, (long long)n - 1);
    const int r = div_by(by_units, i), u = i - r * (int)by_units.d;
    const long long row = (long long)row0 + r;
    if constexpr (WIDE) {
      if (!on) continue;
      float x[8], res[8];
      get8<DT>(a.x.p, row * a.x.stride + 8 * u, x);
      if (a.res.p) get8<DT>(a.res.p, row * a.res.stride + 8 * u, res);
      const uint32_t keep = kept_bits(u, (uint32_t)row, step, a.seed, a.threshold);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = keep >> j & 1 ? x[j] * a.scale : 0.f;
        if (a.res.p) x[j] += res[j];
      }
      if constexpr (DT == EMB_F32) {
        put_unit<DT, 4>(a.y.p, row * a.y.stride + 8 * u, x);
        put_unit<DT, 4>(a.y.p, row * a.y.stride + 8 * u + 4, x + 4);
      } else {
        put_unit<DT, 8>(a.y.p, row * a.y.stride + 8 * u, x);
      }
    } else {
      // element e of the wave's 512 is element e % 8 of lane e / 8's unit
      const uint32_t keep = on ? kept_bits(u, (uint32_t)row, step, a.seed, a.threshold) : 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int src = 8 * k + (lane >> 3), j = lane & 7;
        const int rr = __shfl(r, src, 64), c = 8 * __shfl(u, src, 64) + j;
        const uint32_t bits = __shfl(keep, src, 64);
        if (i0 + src >= n || c >= a.dim) continue;
        const long long at = (long long)row0 + rr;
        float x = bits >> j & 1 ? ld1<DT>(a.x.p, at * a.x.stride + c) * a.scale : 0.f;
        if (a.res.p) x += ld1<DT>(a.res.p, at * a.res.stride + c);
        st1<DT>(const_cast<void*>(a.y.p), at * a.y.stride + c, x);
      }
    }
  }
}

template <int DT>
hipError_t launch_dropout_t(const DropoutArgs& a, bool wide, hipStream_t st) {
  const uint32_t units = (uint32_t)((a.dim + 7ll) / 8);
  const FastDiv by = fast_div(units);
  const long long rows_at_once = std::max<long long>(1, (1ll << 30) / units);
  for (long long r0 = 0; r0 < a.rows; r0 += rows_at_once) {
    const int n = (int)(std::min(rows_at_once, a.rows - r0) * units);
    const unsigned grid = (unsigned)std::min<long long>((n + 255ll) / 256, 1 << 20);
    if (wide) k_dropout<DT, true><<<grid, 256, 0, st>>>(a, by, (uint32_t)r0, n);
    else k_dropout<DT, false><<<grid, 256, 0, st>>>(a, by, (uint32_t)r0, n);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t st) {
  const int E = a.x.dtype == EMB_F32 ? 4 : 8;
  const bool wide = a.dim % E == 0 && fits(a.x, E) && fits(a.y, E);
  int blocks;
  return launch_norm_types<false>(a, a.x.dtype, a.y.dtype, wide, 2048, st, &blocks);
}

int layer_norm_back_blocks(long long rows, int dim) {
  return (int)std::min<long long>(rows, dim <= 1024 ? 1024 : dim <= 4096 ? 512 : 256);
}

hipError_t launch_layer_norm_back(const LayerNormBackArgs& a, hipStream_t st) {
  const int E = a.x.dtype == EMB_F32 ? 4 : 8;
  const bool wide = a.dim % E == 0 && fits(a.x, E) && fits(a.dy, E) && fits(a.dx, E);
  int blocks = 0;
  if (a.rows > 0) {
    if (hipError_t e = launch_norm_types<true>(a, a.x.dtype, a.dy.dtype, wide, layer_norm_back_blocks(a.rows, a.dim), st,
                                               &blocks))
      return e;
  }
  if (a.dw || a.db) k_layer_norm_dw<<<(2 * a.dim + 31) / 32, 1024, 0, st>>>(a.part, blocks, a.dim, a.dw, a.db);
  return hipGetLastError();
}

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t st) {
  const int E = a.x.dtype == EMB_F32 ? 4 : 8;
  const bool wide = a.dim % 8 == 0 && fits(a.x, E) && fits(a.y, E) && (!a.res.p || fits(a.res, E));
  if (a.x.dtype == EMB_F32) return launch_dropout_t<EMB_F32>(a, wide, st);
  if (a.x.dtype == EMB_BF16) return launch_dropout_t<EMB_BF16>(a, wide, st);
  return launch_dropout_t<EMB_F16>(a, wide, st);
}

}  // namespace emb
