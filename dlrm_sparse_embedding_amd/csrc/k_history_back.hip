// Gradient of the attention of histories (k_history.hip).
//
// Mathematics. With P_ij = 2^(s_ij - z_i) and dP_ij = dout_i . v_j,
//     dS_ij = P_ij (dP_ij - sum_j P_ij dP_ij),
//     dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,
//     dv_j = sum_i P_ij dout_i,  dbias[row] = sum of dS_ij over row(i - j) = row.
// The first kernel goes along the keys of 128 queries for dq, the second along
// the queries of 128 keys for dk, dv and dbias: each sum is one wave's, in one
// order, without atomics.
//
// The rows' sums. sum_j P_ij dP_ij is dout_i . out_i but for the rounding of out,
// which is enough for 16-bit results but not for dbias: its fp32 sums cancel (dS
// sums to zero along each row), and the rounding does not. The first kernel
// therefore starts from dout . out, sums its own dS along the row, which gives
// what the start was off by, and hands the corrected sum to the second one, at no
// further product.
//
// Precision. P and dS are fp32 and rounded to the heads' type for the products.
// fp16 ones are scaled first: P by 2^15, dS by a power of two that each column of
// the product keeps for itself, chosen when its first values come and lowered when
// larger ones do, as the running maximum of a softmax is.
#include <algorithm>

#include "history_device.h"

namespace emb {

namespace {

constexpr int kRows = 128;  // rows of a block

struct BackDev {
  HistoryBackArgs a;
  float scale2;
  FastDiv by_m;
  int m, tiles, bias_rows;
};

// A power of two for a lane's column of dS and of the sums that it enters.
template <int DT>
struct ColumnScale {
  float c = DT == EMB_F16 ? 0x1p100f : 1.f;
  // Lowers the column's power of two where |x| would pass 2^14 and rescales acc.
  template <int N>
  __device__ __forceinline__ void fit(const f16v& x, f16v (&acc)[N]) {
    if constexpr (DT == EMB_F16) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
      top = both_halves_max(top);
      const bool down = top * c > 0x1p14f;
      if (__ballot(down)) {
        // the largest becomes 2^9 .. 2^10
        const int e = (int)(__float_as_uint(top) >> 23) - 127;
        const float next = __uint_as_float((uint32_t)max(127 + 9 - e, 1) << 23);
        const float by = down ? next / c : 1.f;
        c = down ? next : c;
#pragma unroll
        for (int d = 0; d < N; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[d][i] *= by;
      }
    }
  }
  __device__ __forceinline__ f16v scaled(const f16v& x) const {
    if constexpr (DT != EMB_F16) return x;
    f16v y;
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = x[i] * c;
    return y;
  }
};

// acc[d] += (columns of 32 rows of `tile`) times w. GUARD: see guarded_product.
template <int DT, int D, bool GUARD>
__device__ __forceinline__ void add_product(f16v (&acc)[D / 32], const short* tile, const s8v (&w)[2], int lo, int hi) {
  if (GUARD && any_special<DT, D>(tile)) {
    guarded_product<DT, D>(acc, tile, 0, w, lo, hi);
    return;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int d = 0; d < D / 32; ++d) acc[d] = mfma<DT>(column_operand<D>(tile, 16 * k, d), w[k], acc[d]);
}

// z of a row in log2 units, so that P = 2^(s - z); +infinity for one that sees nothing.
__device__ __forceinline__ float z_of(float lse) { return lse == kNegInf ? -kNegInf : lse * kLog2e; }

// ---- dq and the rows' sums ------------------------------------------------------

template <int DT, int D>
struct QueryWave {
  s8v q[D / 16], go[D / 16];
  f16v dq[D / 32];
  ColumnScale<DT> c;
  float z, delta, error;  // the row's z, sum of P dP, and this lane's part of what it is off by
};

// 32 keys. EDGE: not every row sees all of them.
template <int DT, int D, bool BIAS, bool EDGE>
__device__ __forceinline__ void dq_step(const BackDev& p, QueryWave<DT, D>& w, const BiasLds& sb, float* win,
                                        const short* ks, const short* vs, int k0, int q0, int seen) {
  const int lane = threadIdx.x & 63;
  Biases b{};
  if (BIAS) b = biases_of(p.a.f.h, sb, q0 + 31 - k0, win);
  f16v s{}, dp{};
#pragma unroll
  for (int i = 0; i < D / 16; ++i) s = mfma<DT>(row_operand<D>(ks, 0, i), w.q[i], s);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) dp = mfma<DT>(row_operand<D>(vs, 0, i), w.go[i], dp);
  if (BIAS && !b.far) {
    const float* at = win + 4 * (lane >> 5) + 31 - (lane & 31);
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], p.scale2, at[8 * (i / 4) + i % 4] - w.z);
  } else {
    const float add = (BIAS ? b.value : 0.f) - w.z;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], p.scale2, add);
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    s[i] = __builtin_amdgcn_exp2f(s[i]) * (dp[i] - w.delta);
    if (EDGE && k0 + 8 * (i / 4) + 4 * (lane >> 5) + i % 4 >= seen) s[i] = 0.f;
    sum += s[i];
  }
  w.error += sum;
  w.c.fit(s, w.dq);
  s8v ds[2];
  pack_tile<DT>(w.c.scaled(s), ds);
  add_product<DT, D, EDGE>(w.dq, ks, ds, 0, seen - k0);
}

template <int DT, int D, bool BIAS>
__global__ __launch_bounds__(256, 2) void k_history_dq(BackDev p) {
  __shared__ __attribute__((aligned(1024))) short s_k[2][kTile * D], s_v[2][kTile * D];
  __shared__ BiasLds s_bias;
  __shared__ float s_win[BIAS ? 4 : 1][64];
  const HistoryArgs& a = p.a.f;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  report_offsets(a.offsets, a.seqs, a.tokens, a.h.error);
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int head = id / p.tiles;
  if (head >= a.h.q_heads) return;
  const SeqTile t = seq_tile(a, p.tiles - 1 - id % p.tiles, kRows);
  if (t.r0 >= t.len) return;
  const int kh = div_by(p.by_m, head);
  const int end = a.h.causal ? min(t.r0 + kRows, t.len) : t.len;
  const uint32_t k_step = 2 * (uint32_t)a.k.ts, v_step = 2 * (uint32_t)a.v.ts;
  const uint64_t k_at = uniform((uint64_t)a.k.p + 2 * (t.first * a.k.ts + kh * a.k.hs));
  const uint64_t v_at = uniform((uint64_t)a.v.p + 2 * (t.first * a.v.ts + kh * a.v.hs));
  const uint32_t lds_k = (uint32_t)(uintptr_t)(lds_elem*)&s_k[0][0], lds_v = (uint32_t)(uintptr_t)(lds_elem*)&s_v[0][0];
  const RowFetch<D> f;
  auto fetch = [&](int k0, int b) {
    f.rows(k_at + (uint64_t)k0 * k_step, k_step, t.len - 1 - k0, lds_k + b * kTile * D * 2);
    f.rows(v_at + (uint64_t)k0 * v_step, v_step, t.len - 1 - k0, lds_v + b * kTile * D * 2);
  };
  fetch(0, 0);
  if (BIAS) {
    stage_bounds(a.h, s_bias);
    stage_bias(a, head, s_bias);
  }
  const int q0 = t.r0 + 32 * wave, place = q0 + (lane & 31);
  const bool live = q0 < t.len;
  const long long token = t.first + min(place, t.len - 1);
  QueryWave<DT, D> w;
  load_operands<D>(a.q, token, head, w.q);
  load_operands<D>(p.a.dout, token, head, w.go);
  {
    s8v o[D / 16];
    load_operands<D>(a.out, token, head, o);
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      float x[8], y[8];
      widen<DT>(__builtin_bit_cast(u4, o[i]), x);
      widen<DT>(__builtin_bit_cast(u4, w.go[i]), y);
#pragma unroll
      for (int j = 0; j < 8; ++j) dot += x[j] * y[j];
    }
    w.delta = both_halves_sum(dot);
  }
  w.z = z_of(a.lse[token * a.h.q_heads + head]);
  w.error = 0.f;
#pragma unroll
  for (int d = 0; d < D / 32; ++d) w.dq[d] = f16v{};
  const int seen = a.h.causal ? min(place + 1, t.len) : t.len;
  const int seen_by_all = a.h.causal ? min(q0 + 1, t.len) : t.len;
  const int seen_by_any = a.h.causal ? min(q0 + 32, t.len) : t.len;
  for (int k0 = 0, b = 0; k0 < end; k0 += kTile, b ^= 1) {
    fetched();
    __syncthreads();
    if (k0 + kTile < end) fetch(k0 + kTile, b ^ 1);
    if (!live) continue;
    float* win = s_win[BIAS ? wave : 0];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int k = k0 + 32 * n;
      const short *ks = s_k[b] + 32 * n * D, *vs = s_v[b] + 32 * n * D;
      if (k + 32 <= seen_by_all) dq_step<DT, D, BIAS, false>(p, w, s_bias, win, ks, vs, k, q0, seen);
      else if (k < seen_by_any) dq_step<DT, D, BIAS, true>(p, w, s_bias, win, ks, vs, k, q0, seen);
    }
  }
  if (!live) return;
  const bool store = place < t.len;
  const float delta = w.delta + both_halves_sum(w.error);
  if (store && lane < 32) p.a.rows[(long long)head * a.tokens + token] = delta;
  short* dst = reinterpret_cast<short*>(const_cast<void*>(p.a.dq.p)) + token * p.a.dq.ts + head * p.a.dq.hs +
               8 * (lane >> 5);
  store_columns<DT, D>(dst, w.dq, a.h.scale / w.c.c, store);
}

// ---- dk, dv and dbias -----------------------------------------------------------

template <int DT, int D>
struct KeyWave {
  s8v k[D / 16], v[D / 16];
  f16v dk[D / 32], dv[D / 32];
  ColumnScale<DT> c;
};

constexpr int kDiag = 40;  // stride of dS in LDS: the lanes' halves, 4 rows apart, lie in different banks

// What the second kernel keeps in LDS for the bias' gradient, a part for each wave.
template <bool BIAS>
struct GradLds {
  float ds[4][32 + 32 * kDiag + 32];
  float sum[4][2 * EMB_MAX_BUCKETS];
};
template <>
struct GradLds<false> {};

// Adds a tile's dS to the sums of its rows of the bias: along its 63 diagonals, a
// lane for each, then over the neighbouring lanes of one row, in a fixed order.
__device__ __forceinline__ void add_diagonals(const f16v& s, int row, float* ds, float* sum) {
  const int lane = threadIdx.x & 63, c = lane & 31;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int i = 0; i < 16; ++i) ds[32 + (8 * (i / 4) + 4 * (lane >> 5) + i % 4) * kDiag + c] = s[i];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  // diagonal x holds (r, c) with 31 - r + c = x
  float v = 0.f;
#pragma unroll 8
  for (int r = 0; r < 32; ++r) {
    const int at = lane - 31 + r;
    const float x = ds[32 + r * kDiag + min(max(at, 0), 31)];
    v += at >= 0 && at < 32 ? x : 0.f;
  }
  if (lane == 63) row = -1;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const float x = __shfl_down(v, d, 64);
    const int r = __shfl_down(row, d, 64);
    if (lane + d < 64 && r == row) v += x;
  }
  const int before = __shfl_up(row, 1, 64);
  if (row >= 0 && (lane == 0 || before != row)) sum[row] += v;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// 32 queries from q0 on. EDGE: not every key is seen by all of them.
template <int DT, int D, bool BIAS, bool EDGE>
__device__ __forceinline__ void dkv_step(const BackDev& p, KeyWave<DT, D>& w, const BiasLds& sb, float* win,
                                         GradLds<BIAS>& g, float (&far)[2], const short* qs, const short* gs,
                                         const float* zs, const float* deltas, int q0, int k0, int len) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), h4 = 4 * (lane >> 5);
  Biases b{};
  if (BIAS) b = biases_of(p.a.f.h, sb, q0 + 31 - k0, win);
  f16v s{}, dp{};
#pragma unroll
  for (int i = 0; i < D / 16; ++i) s = mfma<DT>(row_operand<D>(qs, 0, i), w.k[i], s);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) dp = mfma<DT>(row_operand<D>(gs, 0, i), w.v[i], dp);
  const int key = k0 + (lane & 31);
  // the rows that see the key; none sees one behind the end
  const int first = p.a.f.h.causal ? key - q0 : 0, end = key < len ? len - q0 : 0;
  // diagonal of (r, c): 31 - r + c
  const float* at = win + 31 - h4 + (lane & 31);
#pragma unroll
  for (int i4 = 0; i4 < 16; i4 += 4) {
    const f4 z = *reinterpret_cast<const f4*>(zs + 2 * i4 + h4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float add = !BIAS ? 0.f : b.far ? b.value : at[-(2 * i4 + j)];
      float e = __builtin_amdgcn_exp2f(fmaf(s[i4 + j], p.scale2, add - z[j]));
      if (EDGE) e = 2 * i4 + h4 + j >= first && 2 * i4 + h4 + j < end ? e : 0.f;
      s[i4 + j] = e;
    }
  }
  s8v x[2];
  if constexpr (DT == EMB_F16) {
    f16v y;
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = s[i] * 0x1p15f;
    pack_tile<DT>(y, x);
  } else {
    pack_tile<DT>(s, x);
  }
  add_product<DT, D, EDGE>(w.dv, gs, x, first, end);
#pragma unroll
  for (int i4 = 0; i4 < 16; i4 += 4) {
    const f4 delta = *reinterpret_cast<const f4*>(deltas + 2 * i4 + h4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float e = s[i4 + j] * (dp[i4 + j] - delta[j]);
      if (EDGE) e = 2 * i4 + h4 + j >= first && 2 * i4 + h4 + j < end ? e : 0.f;
      s[i4 + j] = e;
    }
  }
  if constexpr (BIAS) {
    if (p.a.dbias) {
      if (b.far) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) sum += s[i];
        if (b.row < p.a.f.h.buckets.n) far[0] += sum;
        else far[1] += sum;
      } else {
        add_diagonals(s, b.row, g.ds[wave], g.sum[wave]);
      }
    }
  }
  w.c.fit(s, w.dk);
  pack_tile<DT>(w.c.scaled(s), x);
  add_product<DT, D, EDGE>(w.dk, qs, x, first, end);
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
  return x;
}

template <int DT, int D, bool BIAS>
__global__ __launch_bounds__(256, D == 64 ? 2 : 1) void k_history_dkv(BackDev p) {
  __shared__ __attribute__((aligned(1024))) short s_q[2][kTile * D], s_g[2][kTile * D];
  __shared__ __attribute__((aligned(16))) float s_z[2][kTile], s_delta[2][kTile];
  __shared__ BiasLds s_bias;
  __shared__ GradLds<BIAS> s_grad;
  __shared__ float s_win[BIAS ? 4 : 1][64];
  const HistoryArgs& a = p.a.f;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int id = xcd_remap(blockIdx.x, gridDim.x);
  const int kh = id / p.tiles, tile = id % p.tiles;
  if (kh >= a.h.kv_heads) return;
  const SeqTile t = seq_tile(a, tile, kRows);
  const bool grad = BIAS && p.a.dbias;
  float* part = p.a.part + ((long long)tile * a.h.q_heads + kh * p.m) * p.bias_rows;
  if (t.r0 >= t.len) {
    if (grad)
      for (int i = threadIdx.x; i < p.m * p.bias_rows; i += 256) part[i] = 0.f;
    return;
  }
  const int k0 = t.r0 + 32 * wave, place = k0 + (lane & 31);
  const bool live = k0 < t.len;
  const long long token = t.first + min(place, t.len - 1);
  KeyWave<DT, D> w;
  load_operands<D>(a.k, token, kh, w.k);
  load_operands<D>(a.v, token, kh, w.v);
#pragma unroll
  for (int d = 0; d < D / 32; ++d) w.dk[d] = w.dv[d] = f16v{};
  const int begin = a.h.causal ? t.r0 : 0;
  const uint32_t q_step = 2 * (uint32_t)a.q.ts, g_step = 2 * (uint32_t)p.a.dout.ts;
  const uint32_t lds_q = (uint32_t)(uintptr_t)(lds_elem*)&s_q[0][0], lds_g = (uint32_t)(uintptr_t)(lds_elem*)&s_g[0][0];
  const RowFetch<D> f;
  if (BIAS) stage_bounds(a.h, s_bias);
  for (int hh = 0; hh < p.m; ++hh) {
    const int head = kh * p.m + hh;
    const uint64_t q_at = uniform((uint64_t)a.q.p + 2 * (t.first * a.q.ts + head * a.q.hs));
    const uint64_t g_at = uniform((uint64_t)p.a.dout.p + 2 * (t.first * p.a.dout.ts + head * p.a.dout.hs));
    auto fetch = [&](int q0, int b) {
      f.rows(q_at + (uint64_t)q0 * q_step, q_step, t.len - 1 - q0, lds_q + b * kTile * D * 2);
      f.rows(g_at + (uint64_t)q0 * g_step, g_step, t.len - 1 - q0, lds_g + b * kTile * D * 2);
    };
    // z and the rows' sums of a tile, by a thread each
    auto row_values = [&](int q0, int b) {
      if (threadIdx.x < kTile) {
        const long long at = t.first + min(q0 + (int)threadIdx.x, t.len - 1);
        s_z[b][threadIdx.x] = z_of(a.lse[at * a.h.q_heads + head]);
      } else if (threadIdx.x < 2 * kTile) {
        const long long at = t.first + min(q0 + (int)threadIdx.x - kTile, t.len - 1);
        s_delta[b][threadIdx.x - kTile] = p.a.rows[(long long)head * a.tokens + at];
      }
    };
    __syncthreads();  // the last head's tiles and bias are done with
    fetch(begin, 0);
    row_values(begin, 0);
    if (BIAS) stage_bias(a, head, s_bias);
    if constexpr (BIAS) {
      for (int i = threadIdx.x; i < 4 * 2 * EMB_MAX_BUCKETS; i += 256) (&s_grad.sum[0][0])[i] = 0.f;
    }
    float far[2] = {0.f, 0.f};
    for (int q0 = begin, b = 0; q0 < t.len; q0 += kTile, b ^= 1) {
      fetched();
      __syncthreads();
      if (q0 + kTile < t.len) {
        fetch(q0 + kTile, b ^ 1);
        row_values(q0 + kTile, b ^ 1);
      }
      if (!live) continue;
      float* win = s_win[BIAS ? wave : 0];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int q = q0 + 32 * n;
        if (q >= t.len || (a.h.causal && q + 31 < k0)) continue;
        const short *qs = s_q[b] + 32 * n * D, *gs = s_g[b] + 32 * n * D;
        const float *zs = s_z[b] + 32 * n, *deltas = s_delta[b] + 32 * n;
        if (q + 32 <= t.len && (a.h.causal ? q >= k0 + 31 : k0 + 32 <= t.len))
          dkv_step<DT, D, BIAS, false>(p, w, s_bias, win, s_grad, far, qs, gs, zs, deltas, q, k0, t.len);
        else
          dkv_step<DT, D, BIAS, true>(p, w, s_bias, win, s_grad, far, qs, gs, zs, deltas, q, k0, t.len);
      }
    }
    if constexpr (BIAS) {
      if (grad) {
        const float near = wave_sum(far[0]), beyond = wave_sum(far[1]);
        const int n = a.h.buckets.n;
        if (lane == 0) {
          s_grad.sum[wave][n - 1] += near;
          s_grad.sum[wave][2 * n - 1] += beyond;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < p.bias_rows; i += 256)
          part[hh * p.bias_rows + i] = (s_grad.sum[0][i] + s_grad.sum[1][i]) + (s_grad.sum[2][i] + s_grad.sum[3][i]);
      }
    }
  }
  if (!live) return;
  const bool store = place < t.len;
  short* dk = reinterpret_cast<short*>(const_cast<void*>(p.a.dk.p)) + token * p.a.dk.ts + kh * p.a.dk.hs + 8 * (lane >> 5);
  short* dv = reinterpret_cast<short*>(const_cast<void*>(p.a.dv.p)) + token * p.a.dv.ts + kh * p.a.dv.hs + 8 * (lane >> 5);
  store_columns<DT, D>(dk, w.dk, a.h.scale / w.c.c, store);
  store_columns<DT, D>(dv, w.dv, DT == EMB_F16 ? 0x1p-15f : 1.f, store);
}

// The bias' gradient from the tiles' partial sums, in 64 bits: a block for each
// row and head.
__global__ __launch_bounds__(256) void k_history_dbias(const float* __restrict__ part, int tiles, int heads, int rows,
                                                       float* __restrict__ dbias) {
  __shared__ double s[4];
  const int row = blockIdx.x % rows, head = blockIdx.x / rows;
  double acc = 0.0;
  for (int t = threadIdx.x; t < tiles; t += 256) acc += (double)part[((long long)t * heads + head) * rows + row];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) acc += __shfl_xor(acc, d, 64);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = acc;
  __syncthreads();
  if (threadIdx.x == 0) dbias[(long long)row * heads + head] = (float)(s[0] + s[1] + s[2] + s[3]);
}

template <int DT, int D, bool BIAS>
hipError_t launch(const BackDev& p, hipStream_t st) {
  const HistoryView& h = p.a.f.h;
  const long long tiles = p.tiles;
  if (p.a.f.tokens == 0) {
    k_history_dbias<<<(unsigned)(p.bias_rows * h.q_heads), 256, 0, st>>>(nullptr, 0, h.q_heads, p.bias_rows, p.a.dbias);
    return hipGetLastError();
  }
  k_history_dq<DT, D, BIAS><<<(unsigned)((tiles * h.q_heads + 7) / 8 * 8), 256, 0, st>>>(p);
  if (hipError_t e = hipGetLastError()) return e;
  k_history_dkv<DT, D, BIAS><<<(unsigned)((tiles * h.kv_heads + 7) / 8 * 8), 256, 0, st>>>(p);
  if (hipError_t e = hipGetLastError()) return e;
  if (BIAS && p.a.dbias) {
    k_history_dbias<<<(unsigned)(p.bias_rows * h.q_heads), 256, 0, st>>>(p.a.part, p.tiles, h.q_heads, p.bias_rows,
                                                                        p.a.dbias);
    return hipGetLastError();
  }
  return hipSuccess;
}

template <int DT>
hipError_t launch_t(const BackDev& p, hipStream_t st) {
  const bool bias = p.a.f.bias != nullptr;
  switch (p.a.f.h.dim) {
    case 64: return bias ? launch<DT, 64, true>(p, st) : launch<DT, 64, false>(p, st);
    case 96: return bias ? launch<DT, 96, true>(p, st) : launch<DT, 96, false>(p, st);
    default: return bias ? launch<DT, 128, true>(p, st) : launch<DT, 128, false>(p, st);
  }
}

}  // namespace

HistoryBackPlan history_back_plan(const HistoryView& h, long long tokens, int seqs) {
  HistoryBackPlan p{};
  const long long rows = h.buckets.n * (h.causal ? 1 : 2);
  p.part_off = ((size_t)tokens * h.q_heads * 4 + 255) & ~size_t(255);
  p.bytes = p.part_off + (size_t)(seq_tiles(tokens, seqs, kRows) * h.q_heads * rows * 4);
  return p;
}

hipError_t launch_history_back(const HistoryBackArgs& a, hipStream_t st) {
  BackDev p{};
  p.a = a;
  p.scale2 = a.f.h.scale * kLog2e;
  p.m = a.f.h.q_heads / a.f.h.kv_heads;
  p.by_m = fast_div((uint32_t)p.m);
  p.tiles = (int)seq_tiles(a.f.tokens, a.f.seqs, kRows);
  p.bias_rows = a.f.h.buckets.n * (a.f.h.causal ? 1 : 2);
  return a.f.h.dtype == EMB_BF16 ? launch_t<EMB_BF16>(p, st) : launch_t<EMB_F16>(p, st);
}

}  // namespace emb
