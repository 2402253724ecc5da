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
// Measured: fp32 rows of 262144 x 128 normed to bf16 36 us (5.6 TB/s); gradient of
// 24577 x 1024 bf16 30 us (5.0 TB/s) and 4 for the weights' sums over the blocks;
// dropout and sum of 32768 x 1024 bf16 35 us (5.8 TB/s): its Philox draw for eight
// elements, and a second one where bits tie (one unit of eight in 8000), fit beside
// the memory's time. Gradient of fp32 rows with 16-bit dy, as a table's are: 262144
// x 128 66 us (5.1 TB/s), 24577 x 512 31 us (4.1 TB/s, 24 without the weights' sums).
// Beyond 1024 columns it is further off: 6000 x 4096 bf16 47 us (3.1 TB/s), for the
// barriers of a row's waves and, in blocks of 1024 threads, 128 registers, which do
// not hold a row without spilling 4 to 15; off 16-byte borders 16 to 57.
//
// Layout. A row belongs to a group of G lanes (a power of two, at most a wave)
// or, beyond 1024 columns, to 4 or 16 waves; lane u holds the columns E (k G + u) ..
// + E - 1, k < K: each access of the group is one run of 16 bytes a lane (8 on the
// 16-bit side of fp32 rows).
#include <algorithm>

#include "seq_device.h"

namespace emb {

namespace {

typedef unsigned long long u64;

// E neighbouring elements as they lie in memory. Fully aligned units (ANY = 0)
// are whole, read and written once, and go past the L2; others are accesses of
// the same width on any element's address, which the hardware splits (24577 x
// 1001 bf16: norm 91 -> 48 us against single elements), and leave what they
// share of lines to the L2.
template <int DT, int E>
struct Unit {
  using T = typename Elem<DT>::T;
  static constexpr int kWords = E * sizeof(T) / 4;
  static_assert(kWords == 2 || kWords == 4, "8 or 16 bytes");
  typedef uint32_t V __attribute__((ext_vector_type(kWords)));
  typedef uint32_t VU __attribute__((ext_vector_type(kWords), aligned(sizeof(T))));
};
template <int DT, int E>
using UnitV = typename Unit<DT, E>::V;

// The first n (at least 1; ANY = 0: all E) from element i on.
template <int DT, int E, bool ANY>
__device__ __forceinline__ UnitV<DT, E> get_unit(const void* p, long long i, int n) {
  using U = Unit<DT, E>;
  const typename U::T* at = reinterpret_cast<const typename U::T*>(p) + i;
  if constexpr (!ANY) {
    return __builtin_nontemporal_load(reinterpret_cast<const typename U::V*>(at));
  } else {
    typename U::V v{};
    if (n == E) {
      v = *reinterpret_cast<const typename U::VU*>(at);
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(at);
      const uint32_t* f = reinterpret_cast<const uint32_t*>(at);
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (j < n) {
          if constexpr (DT == EMB_F32) v[j] = f[j];
          else v[j / 2] |= (uint32_t)h[j] << 16 * (j % 2);
        }
    }
    return v;
  }
}
template <int DT, int E>
__device__ __forceinline__ void widen_unit(const UnitV<DT, E> v, float* out) {
  if constexpr (Unit<DT, E>::kWords == 4) {
    widen<DT>(v, out);
  } else {
    float f[8];
    widen<DT>(u4{v.x, v.y, 0, 0}, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = f[j];
  }
}
template <int DT, int E, bool ANY>
__device__ __forceinline__ void put_unit(const void* p, long long i, int n, const float* in) {
  using U = Unit<DT, E>;
  typename U::T* at = reinterpret_cast<typename U::T*>(const_cast<void*>(p)) + i;
  if (ANY && n < E) {
#pragma unroll
    for (int j = 0; j < E; ++j)
      if (j < n) st1<DT>(const_cast<void*>(p), i + j, in[j]);
    return;
  }
  typename U::V v;
  if constexpr (U::kWords == 4) {
    v = narrow<DT>(in);
  } else {
    const float f[8] = {in[0], in[1], in[2], in[3]};
    const u4 x = narrow<DT>(f);
    v = u2{x.x, x.y};
  }
  if constexpr (ANY) *reinterpret_cast<typename U::VU*>(at) = v;
  else __builtin_nontemporal_store(v, reinterpret_cast<typename U::V*>(at));
}

// The lanes of a row.
template <int E, int K, bool BIG, bool ANY>
struct Place {
  int u, width, dim;  // this lane, how many there are, columns
  int per, group;     // rows a block takes at once, and which of them is this lane's
  __device__ __forceinline__ Place(int G, int columns) {
    u = threadIdx.x & (G - 1);
    width = G;
    dim = columns;
    per = blockDim.x / G;
    group = threadIdx.x / G;
  }
  __device__ __forceinline__ int col(int k) const { return E * (k * width + u); }
  // columns of unit k
  __device__ __forceinline__ int count(int k) const {
    return ANY ? max(0, min(dim - col(k), E)) : col(k) < dim ? E : 0;
  }
  // Clears unit k's elements behind the row's end. Few lanes have a part of a
  // unit; that the compiler does not know their count keeps it from holding a
  // mask for every element.
  __device__ __forceinline__ void clear(int k, float* x) const {
    int n = count(k);
    if (ANY && n > 0 && n < E) {
      asm volatile("" : "+v"(n));
#pragma unroll
      for (int j = 0; j < E; ++j) x[j] = j < n ? x[j] : 0.f;
    }
#pragma unroll
    for (int j = 0; j < E; ++j) x[j] = n > 0 ? x[j] : 0.f;
  }
};

// Sum over the row's lanes, in one order for all of them; `turn` alternates
// between a block's uses of it. Steps that go beyond the row add nothing.
template <bool BIG>
__device__ __forceinline__ float row_sum(float x, int G, int turn, float (*s)[16]) {
  typedef unsigned u2v __attribute__((ext_vector_type(2)));
  auto add = [&](float y, int above) { x += BIG || G > above ? y : 0.f; };
  add(dpp<0xB1>(x), 1);   // swap neighbours
  add(dpp<0x4E>(x), 2);   // swap pairs
  add(dpp<0x141>(x), 4);  // mirror 8 lanes: quads are uniform by now
  add(dpp<0x140>(x), 8);  // mirror 16 lanes
  const uint32_t b = __float_as_uint(x);
  const u2v r = __builtin_amdgcn_permlane16_swap(b, b, false, false);
  x = BIG || G > 16 ? __uint_as_float(r.x) + __uint_as_float(r.y) : x;
  const uint32_t c = __float_as_uint(x);
  const u2v q = __builtin_amdgcn_permlane32_swap(c, c, false, false);
  x = BIG || G > 32 ? __uint_as_float(q.x) + __uint_as_float(q.y) : x;
  if constexpr (BIG) {
    if ((threadIdx.x & 63) == 0) s[turn][threadIdx.x >> 6] = x;
    __syncthreads();
    // the row's waves, 4 or 16 of them, by as many lanes
    const int waves = G >> 6;
    x = s[turn][threadIdx.x / G * waves + (threadIdx.x & (waves - 1))];
    x += dpp<0xB1>(x);
    x += dpp<0x4E>(x);
    const float y = dpp<0x141>(x);
    x += waves > 4 ? y : 0.f;
    const float z = dpp<0x140>(x);
    x += waves > 4 ? z : 0.f;
  }
  return x;
}

// A row as it lies in memory. Lanes and rows without columns of their own read
// others (nothing of them is used), so that all loads go out at once.
template <int DT, int E, int K, bool BIG, bool ANY>
__device__ __forceinline__ void get_row(const Place<E, K, BIG, ANY>& at, const Rows2D& r, long long row, long long rows,
                                        UnitV<DT, E> (&v)[K]) {
  const long long i = min(row, rows - 1) * r.stride;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const bool none = at.count(k) == 0;
    v[k] = get_unit<DT, E, ANY>(r.p, i + (none ? 0 : at.col(k)), none ? min(at.dim, E) : at.count(k));
  }
}
template <int DT, int E, int K, bool BIG, bool ANY>
__device__ __forceinline__ void widen_row(const Place<E, K, BIG, ANY>& at, const UnitV<DT, E> (&v)[K],
                                          float (&x)[K * E]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    widen_unit<DT, E>(v[k], x + k * E);
    if (at.count(k) == 0) {
#pragma unroll
      for (int j = 0; j < E; ++j) x[k * E + j] = 0.f;
    }
  }
}
template <int DT, int E, int K, bool BIG, bool ANY>
__device__ __forceinline__ void put_row(const Place<E, K, BIG, ANY>& at, const Rows2D& r, long long row,
                                        const float (&x)[K * E]) {
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (at.count(k) > 0) put_unit<DT, E, ANY>(r.p, row * r.stride + at.col(k), at.count(k), x + k * E);
}
// The lane's part of a weight (`none` where there is none); anything behind the
// row's end.
template <int E, int K, bool BIG, bool ANY>
__device__ __forceinline__ void get_weight(const Place<E, K, BIG, ANY>& at, const float* w, float none,
                                           float (&out)[K * E]) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (!w) {
#pragma unroll
      for (int j = 0; j < E; ++j) out[k * E + j] = none;
    } else if (!ANY || at.count(k) == E) {
      const float* from = w + (at.count(k) ? at.col(k) : 0);  // lanes behind the end read its start
#pragma unroll
      for (int j = 0; j < E; j += 4) load4<EMB_F32>(from + j, out + k * E + j);
    } else {
#pragma unroll
      for (int j = 0; j < E; ++j) out[k * E + j] = w[min(at.col(k) + j, at.dim - 1)];
    }
  }
}

// x becomes the differences from the row's mean (0 behind its end); the
// reciprocal deviation.
template <int E, int K, bool BIG, bool ANY>
__device__ __forceinline__ float center(const Place<E, K, BIG, ANY>& at, float (&x)[K * E], float eps, int G,
                                        float (*s)[16]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < K * E; ++i) sum += x[i];
  const float mean = row_sum<BIG>(sum, G, 0, s) / (float)at.dim;
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
#pragma unroll
    for (int j = 0; j < E; ++j) x[k * E + j] -= mean;
    at.clear(k, x + k * E);
#pragma unroll
    for (int j = 0; j < E; ++j) ss += x[k * E + j] * x[k * E + j];
  }
  return 1.f / sqrtf(row_sum<BIG>(ss, G, 1, s) / (float)at.dim + eps);
}

template <int XT, int YT, int E, int K, bool BIG, bool ANY>
__global__ __launch_bounds__(BIG ? 1024 : 256) void k_layer_norm(LayerNormArgs a, int G) {
  __shared__ float s[2][16];
  const Place<E, K, BIG, ANY> at(G, a.dim);
  const long long step = (long long)gridDim.x * at.per;
  long long row = (long long)blockIdx.x * at.per + at.group;
  UnitV<XT, E> next[K];
  get_row<XT>(at, a.x, row, a.rows, next);
  float w[K * E], b[K * E];
  get_weight(at, a.w, 1.f, w);
  get_weight(at, a.b, 0.f, b);
  // whole blocks stay in the loop: lanes and waves of several rows meet in row_sum
  for (long long row0 = row - at.group; row0 < a.rows; row0 += step, row += step) {
    float x[K * E];
    widen_row<XT>(at, next, x);
    if (row0 + step < a.rows) get_row<XT>(at, a.x, row + step, a.rows, next);
    const float r = center(at, x, a.eps, G, s);
#pragma unroll
    for (int j = 0; j < K * E; ++j) x[j] = x[j] * r * w[j] + b[j];
    if (row < a.rows) put_row<YT>(at, a.y, row, x);
  }
}

// The gradient's blocks have 16 waves, so that their partial sums are few.
constexpr int kBackThreads = 1024;

template <int XT, int YT, int E, int K, bool BIG, bool ANY>
__global__ __launch_bounds__(kBackThreads) void k_layer_norm_back(LayerNormBackArgs a, int G) {
  __shared__ float s[2][16];
  __shared__ float s2[2][16];
  __shared__ float s_part[4 * 2 * 1024];  // 4 of up to 1024 columns or one of up to 4096
  const Place<E, K, BIG, ANY> at(G, a.dim);
  const long long step = (long long)gridDim.x * at.per;
  long long row = (long long)blockIdx.x * at.per + at.group;
  // aligned 16-bit rows are fetched one ahead; others would not fit the registers
  constexpr bool AHEAD = E == 8 && !ANY;
  UnitV<XT, E> next_x[K];
  UnitV<YT, E> next_dy[K];
  if (AHEAD) {
    get_row<XT>(at, a.x, row, a.rows, next_x);
    get_row<YT>(at, a.dy, row, a.rows, next_dy);
  }
  float dw[K * E] = {}, db[K * E] = {};
  for (long long row0 = row - at.group; row0 < a.rows; row0 += step, row += step) {
    if (!AHEAD) {
      get_row<XT>(at, a.x, row, a.rows, next_x);
      get_row<YT>(at, a.dy, row, a.rows, next_dy);
    }
    float x[K * E], dy[K * E];
    widen_row<XT>(at, next_x, x);
    widen_row<YT>(at, next_dy, dy);
    if (AHEAD && row0 + step < a.rows) {
      get_row<XT>(at, a.x, row + step, a.rows, next_x);
      get_row<YT>(at, a.dy, row + step, a.rows, next_dy);
    }
    const float r = center(at, x, a.eps, G, s);
    const bool live = row < a.rows;
    float sg = 0.f, sgh = 0.f;
    float w[K * E];
    const float* from = a.w;
    asm volatile("" : "+s"(from));  // read again for each row, from the caches: no registers for it meanwhile
    get_weight(at, from, 1.f, w);
#pragma unroll
    for (int j = 0; j < K * E; ++j) {
      x[j] *= r;  // h
      dw[j] += live ? dy[j] * x[j] : 0.f;
      db[j] += live ? dy[j] : 0.f;
      dy[j] *= w[j];  // g
      sg += dy[j];
      sgh += dy[j] * x[j];
    }
    const float mg = row_sum<BIG>(sg, G, 0, s2) / (float)a.dim;
    const float mgh = row_sum<BIG>(sgh, G, 1, s2) / (float)a.dim;
#pragma unroll
    for (int j = 0; j < K * E; ++j) x[j] = r * (dy[j] - mg - x[j] * mgh);
    if (live) put_row<XT>(at, a.dx, row, x);
  }
  if (!a.dw && !a.db) return;
  float* part = a.part + (long long)blockIdx.x * 2 * a.dim;
  if (BIG && at.per == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int j = 0; j < E; ++j)
        if (j < at.count(k)) {
          part[at.col(k) + j] = dw[k * E + j];
          part[a.dim + at.col(k) + j] = db[k * E + j];
        }
    return;
  }
  // the wave's rows, then the waves of four arrays at a time (BIG: one), in turn
  if (!BIG) {
    for (int d = G; d < 64; d <<= 1)
#pragma unroll
      for (int j = 0; j < K * E; ++j) {
        dw[j] += __shfl_xor(dw[j], d, 64);
        db[j] += __shfl_xor(db[j], d, 64);
      }
  }
  constexpr int kArrays = BIG ? 1 : 4, kColumns = BIG ? 4096 : 1024;
  const int member = BIG ? at.group : threadIdx.x >> 6;
  for (int turn = 0; turn < (BIG ? at.per : kBackThreads / 64) / kArrays; ++turn) {
    if (member / kArrays == turn && (BIG || (threadIdx.x & 63) < G)) {
      float* mine = s_part + member % kArrays * 2 * kColumns;
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < E; ++j)
          if (j < at.count(k)) {
            const int c = at.col(k) + j;
            mine[c] = (turn ? mine[c] : 0.f) + dw[k * E + j];
            mine[kColumns + c] = (turn ? mine[kColumns + c] : 0.f) + db[k * E + j];
          }
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < 2 * a.dim; i += kBackThreads) {
    const int c = i >= a.dim ? kColumns + i - a.dim : i;
    float t = s_part[c];
#pragma unroll
    for (int n = 1; n < kArrays; ++n) t += s_part[n * 2 * kColumns + c];
    part[i] = t;
  }
}

// Weights' gradients from the blocks' partial sums, in 64 bits: 32 columns for a
// block (whole lines), 32 rows of them at a time, 8 times under way.
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

// How a call's rows are laid out on lanes: 16 elements a lane at most, one unit
// a lane where that leaves no more than 8 lanes. Beyond 1024 columns a row has
// several waves.
struct Shape {
  int K, G, threads;  // G lanes a row
  bool big;
};
Shape shape_of(int dim, int E, int threads) {
  Shape s{};
  const int kmax = 16 / E, units = (dim + E - 1) / E;
  if (dim > 1024) {
    s.big = true;
    s.K = kmax;
    s.G = dim <= 4096 ? 256 : 1024;
    s.threads = std::max(threads, s.G);
    return s;
  }
  s.threads = threads;
  s.K = units <= 8 ? 1 : kmax;
  s.G = 1;
  while (s.G * s.K < units) s.G *= 2;
  return s;
}

template <int XT, int YT, bool BACK, typename A>
hipError_t launch_norm(const A& a, bool any, int cap, hipStream_t st, int* blocks) {
  constexpr int E = XT == EMB_F32 || YT == EMB_F32 ? 4 : 8;
  const Shape s = shape_of(a.dim, E, BACK ? kBackThreads : 256);
  const int per = s.threads / s.G;
  *blocks = (int)std::min<long long>((a.rows + per - 1) / per, cap);
  auto run = [&](auto kernel) { kernel<<<*blocks, s.threads, 0, st>>>(a, s.G); };
#define EMB_NORM(K, BIG, ANY)                                           \
  do {                                                                  \
    if constexpr (BACK) run(k_layer_norm_back<XT, YT, E, K, BIG, ANY>); \
    else run(k_layer_norm<XT, YT, E, K, BIG, ANY>);                     \
  } while (0)
  if (any) {
    if (s.big) EMB_NORM(16 / E, true, true);
    else EMB_NORM(16 / E, false, true);
  } else {
    if (s.big) EMB_NORM(16 / E, true, false);
    else if (s.K == 1) EMB_NORM(1, false, false);
    else EMB_NORM(16 / E, false, false);
  }
#undef EMB_NORM
  return hipGetLastError();
}

template <bool BACK, typename A>
hipError_t launch_norm_types(const A& a, int xt, int yt, bool any, int cap, hipStream_t st, int* blocks) {
  if (xt == EMB_BF16) return launch_norm<EMB_BF16, EMB_BF16, BACK>(a, any, cap, st, blocks);
  if (xt == EMB_F16) return launch_norm<EMB_F16, EMB_F16, BACK>(a, any, cap, st, blocks);
  if (yt == EMB_F32) return launch_norm<EMB_F32, EMB_F32, BACK>(a, any, cap, st, blocks);
  if (yt == EMB_BF16) return launch_norm<EMB_F32, EMB_BF16, BACK>(a, any, cap, st, blocks);
  return launch_norm<EMB_F32, EMB_F16, BACK>(a, any, cap, st, blocks);
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

// The first n of 8 elements.
template <int DT, bool ANY>
__device__ __forceinline__ void get8(const Rows2D& r, long long row, int c, int n, float* x) {
  const long long i = row * r.stride + c;
  if constexpr (DT == EMB_F32) {
    const u4 lo = get_unit<DT, 4, ANY>(r.p, i, min(n, 4));
    u4 hi{};
    if (n > 4) hi = get_unit<DT, 4, ANY>(r.p, i + 4, n - 4);
    widen_unit<DT, 4>(lo, x);
    widen_unit<DT, 4>(hi, x + 4);
  } else {
    widen_unit<DT, 8>(get_unit<DT, 8, ANY>(r.p, i, n), x);
  }
}

// n units of 8 columns from row row0 on, one for each lane at a time.
template <int DT, bool ANY>
__global__ __launch_bounds__(256) void k_dropout(DropoutArgs a, FastDiv by_units, uint32_t row0, int n) {
  const u64 step = a.step ? (u64)*a.step : 0;
  for (long long at = (long long)blockIdx.x * 256 + threadIdx.x; at < n; at += (long long)gridDim.x * 256) {
    const int i = (int)at, r = div_by(by_units, i), u = i - r * (int)by_units.d;
    const int count = ANY ? min(8, a.dim - 8 * u) : 8;
    const long long row = (long long)row0 + r;
    float x[8] = {}, res[8] = {};
    get8<DT, ANY>(a.x, row, 8 * u, count, x);
    if (a.res.p) get8<DT, ANY>(a.res, row, 8 * u, count, res);
    const uint32_t keep = kept_bits(u, (uint32_t)row, step, a.seed, a.threshold);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = keep >> j & 1 ? x[j] * a.scale : 0.f;
      if (a.res.p) x[j] += res[j];
    }
    const long long o = row * a.y.stride + 8 * u;
    if constexpr (DT == EMB_F32) {
      put_unit<DT, 4, ANY>(a.y.p, o, min(count, 4), x);
      if (count > 4) put_unit<DT, 4, ANY>(a.y.p, o + 4, count - 4, x + 4);
    } else {
      put_unit<DT, 8, ANY>(a.y.p, o, count, x);
    }
  }
}

template <int DT>
hipError_t launch_dropout_t(const DropoutArgs& a, bool any, hipStream_t st) {
  const uint32_t units = (uint32_t)((a.dim + 7ll) / 8);
  const FastDiv by = fast_div(units);
  const long long rows_at_once = std::max<long long>(1, (1ll << 30) / units);
  for (long long r0 = 0; r0 < a.rows; r0 += rows_at_once) {
    const int n = (int)(std::min(rows_at_once, a.rows - r0) * units);
    const unsigned grid = (unsigned)std::min<long long>((n + 255ll) / 256, 1 << 20);
    if (any) k_dropout<DT, true><<<grid, 256, 0, st>>>(a, by, (uint32_t)r0, n);
    else k_dropout<DT, false><<<grid, 256, 0, st>>>(a, by, (uint32_t)r0, n);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t st) {
  const int E = a.x.dtype == EMB_F32 ? 4 : 8;
  const bool any = a.dim % E != 0 || !fits(a.x, E) || !fits(a.y, E);
  int blocks;
  return launch_norm_types<false>(a, a.x.dtype, a.y.dtype, any, 2048, st, &blocks);
}

int layer_norm_back_blocks(long long rows) { return (int)std::min<long long>(rows, 256); }

hipError_t launch_layer_norm_back(const LayerNormBackArgs& a, hipStream_t st) {
  const int E = a.x.dtype == EMB_F32 ? 4 : 8;
  const bool any = a.dim % E != 0 || !fits(a.x, E) || !fits(a.dy, E) || !fits(a.dx, E);
  int blocks = 0;
  if (a.rows > 0) {
    if (hipError_t e = launch_norm_types<true>(a, a.x.dtype, a.dy.dtype, any, layer_norm_back_blocks(a.rows), st,
                                               &blocks))
      return e;
  }
  if (a.dw || a.db) k_layer_norm_dw<<<(2 * a.dim + 31) / 32, 1024, 0, st>>>(a.part, blocks, a.dim, a.dw, a.db);
  return hipGetLastError();
}

hipError_t launch_dropout(const DropoutArgs& a, hipStream_t st) {
  const int E = a.x.dtype == EMB_F32 ? 4 : 8;
  const bool any = a.dim % 8 != 0 || !fits(a.x, E) || !fits(a.y, E) || (a.res.p && !fits(a.res, E));
  if (a.x.dtype == EMB_F32) return launch_dropout_t<EMB_F32>(a, any, st);
  if (a.x.dtype == EMB_BF16) return launch_dropout_t<EMB_BF16>(a, any, st);
  return launch_dropout_t<EMB_F16>(a, any, st);
}

}  // namespace emb
