// Gradient of the attention of histories (k_history.hip).
//
// Mathematics. With P_ij = 2^(s_ij - z_i) and dP_ij = dout_i . v_j,
//     dS_ij = P_ij (dP_ij - sum_j P_ij dP_ij),
//     dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,
//     dv_j = sum_i P_ij dout_i,  dbias[row] = sum of dS_ij over row(i - j) = row.
// The first kernel goes along the keys of 128 queries for dq, the second along
// the queries of 64 keys for dk, dv and dbias: each sum is one wave's or two's, in
// one order, without atomics.
//
// Bound by vector work and waits between products: 12289 items, 16 x 4 heads of
// 128 bf16, causal: 1180 us (495 TFLOP/s of the five products that it needs; eight
// are made), 1608 with the bias' gradient, 1444 without that but with a bias; dq
// is about 490 of them. Heads of 64: 628 us; 128 users of up to 620 items, 8 x 2
// heads: 389 with the bias' gradient, 332 without, 258 without a bias. Two blocks
// a CU are worth more than registers: dq of 128-wide heads, which spills 9 (bf16) to
// 25 registers (fp16 with a bias) and fetches a few of them back in its loop, took
// 150 us less than with one block and none. dk and dv of 128-wide bf16 heads with a
// bias spill 35 outside the loop over the tiles, of 64-wide fp16 ones with a bias 5.
//
// The rows' sums. sum_j P_ij dP_ij is dout_i . out_i but for the rounding of out,
// which is enough for 16-bit results but not for dbias: its fp32 sums cancel (dS
// sums to zero along each row), and the rounding does not. The first kernel
// therefore starts from dout . out, sums its own dS along the row, which gives e,
// what the start was off by, hands the corrected sum to the second one, and takes
// e sum_j P_ij k_j, one product more, off dq (bf16 heads of 64: dq's error against
// 64 bits 2.5e-3 without it, where rounding the result alone makes 1.7e-3).
//
// Precision. P and dS are fp32 and rounded to the heads' type for the products.
// fp16 ones are scaled first: P by 2^15, dS by a power of two that each column of
// the product keeps for itself, chosen when its first values come and lowered when
// larger ones do, as the running maximum of a softmax is.
#include <algorithm>

#include "history_device.h"

namespace emb {

namespace {

constexpr int kRows = 128;  // queries of a block for dq, and of a tile for dk and dv
constexpr int kKeys = 64;   // keys of a block for dk and dv

struct BackDev {
  HistoryBackArgs a;
  float scale2;
  FastDiv by_m, by_heads, by_kv_heads;
  int m, q_tiles, k_tiles, bias_rows;
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

// z of a row in log2 units, so that P = 2^(s - z); +infinity for one that sees nothing.
__device__ __forceinline__ float z_of(float lse) { return lse == kNegInf ? -kNegInf : lse * kLog2e; }

// ---- dq and the rows' sums ------------------------------------------------------

template <int DT, int D>
struct QueryWave {
  s8v q[D / 16], go[D / 16];
  f16v dq[D / 32];
  f16v pk[D / 32];  // sum P k (fp16: times 2^15)
  ColumnScale<DT> c;
  float z, delta, error;  // the row's z, dout . out, and this lane's part of what that is off by
};

// P packed for a product; fp16 times 2^15 (P is at most 1 but for rounding).
template <int DT>
__device__ __forceinline__ void pack_weights(const f16v& p, s8v (&x)[2]) {
  if constexpr (DT == EMB_F16) {
    f16v y;
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = p[i] * 0x1p15f;
    pack_tile<DT>(y, x);
  } else {
    pack_tile<DT>(p, x);
  }
}

// How many pieces of a lane's dout stay in LDS: with a bias and 128-wide heads there
// are that many registers too few, and a spilled one is fetched by a load that waits
// for the tile in flight (12289 items bf16, with dbias 1657 -> 1616 us).
template <int D, bool BIAS>
constexpr int kHeld = BIAS && D == 128 ? 3 : 0;

// P and dS of 32 keys, packed. edge: not every row sees all of them.
template <int DT, int D, bool BIAS>
__device__ __forceinline__ void dq_weights(const BackDev& p, QueryWave<DT, D>& w, const s8v (*held)[256],
                                           const BiasLds& sb, float* win,
                                           const TileLane<D>& tl, const short* ks, const short* vs, int k0, int q0,
                                           int seen, bool edge, s8v (&xp)[2], s8v (&xs)[2]) {
  const int lane = threadIdx.x & 63;
  Biases b{};
  if (BIAS) b = biases_of(p.a.f.h, sb, q0 + 31 - k0, win);
  f16v s{}, dp{};
#pragma unroll
  for (int i = 0; i < D / 16; ++i) s = mfma<DT>(tl.rows(ks, 0, i), w.q[i], s);
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
    dp = mfma<DT>(tl.rows(vs, 0, i), i < kHeld<D, BIAS> ? held[i][threadIdx.x] : w.go[i], dp);
  if (BIAS && !b.far) {
    const float* at = win + 4 * (lane >> 5) + 31 - (lane & 31);
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], p.scale2, at[8 * (i / 4) + i % 4] - w.z);
  } else {
    const float add = (BIAS ? b.value : 0.f) - w.z;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = fmaf(s[i], p.scale2, add);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    s[i] = __builtin_amdgcn_exp2f(s[i]);
    dp[i] = s[i] * (dp[i] - w.delta);
  }
  if (edge) {
    const uint32_t bits = row_bits(0, seen - k0);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = where_bit(bits, i, s[i]);
      dp[i] = where_bit(bits, i, dp[i]);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) sum += dp[i];
  w.error += sum;
  w.c.fit(dp, w.dq);
  pack_weights<DT>(s, xp);
  pack_tile<DT>(w.c.scaled(dp), xs);
}

template <int DT, int D, bool BIAS>
__global__ __launch_bounds__(256, 2) void k_history_dq(BackDev p) {
  __shared__ __attribute__((aligned(1024))) short s_k[2][kTile * D], s_v[2][kTile * D];
  __shared__ BiasLds s_bias;
  __shared__ float s_win[BIAS ? 4 : 1][64];
  __shared__ s8v s_held[kHeld<D, BIAS> > 0 ? kHeld<D, BIAS> : 1][256];
  const HistoryArgs& a = p.a.f;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  report_offsets(a.offsets, a.seqs, a.tokens, a.h.error);
  int head, tile;
  head_and_tile(blockIdx.x, a.h.q_heads, p.by_heads, &head, &tile);
  const SeqTile t = seq_tile(a, p.q_tiles - 1 - tile, kRows);  // later tiles, which see more, first
  if (t.r0 >= t.len) return;
  const int kh = div_by(p.by_m, head);
  const int end = a.h.causal ? min(t.r0 + kRows, t.len) : t.len;
  const uint32_t k_step = 2 * (uint32_t)a.k.ts, v_step = 2 * (uint32_t)a.v.ts;
  const uint64_t k_at = uniform((uint64_t)a.k.p + 2 * (t.first * a.k.ts + kh * a.k.hs));
  const uint64_t v_at = uniform((uint64_t)a.v.p + 2 * (t.first * a.v.ts + kh * a.v.hs));
  const uint32_t lds_k = (uint32_t)(uintptr_t)(lds_elem*)&s_k[0][0], lds_v = (uint32_t)(uintptr_t)(lds_elem*)&s_v[0][0];
  const RowFetch<D> f;
  auto fetch = [&](int k0, int b) {
    f.rows(k_at + (uint64_t)k0 * k_step, k_step, 0, t.len - 1 - k0, lds_k + b * kTile * D * 2);
    f.rows(v_at + (uint64_t)k0 * v_step, v_step, 0, t.len - 1 - k0, lds_v + b * kTile * D * 2);
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
#pragma unroll
  for (int i = 0; i < kHeld<D, BIAS>; ++i) s_held[i][threadIdx.x] = w.go[i];  // each lane reads its own
  w.z = z_of(a.lse[token * a.h.q_heads + head]);
  w.error = 0.f;
#pragma unroll
  for (int d = 0; d < D / 32; ++d) w.dq[d] = w.pk[d] = f16v{};
  const TileLane<D> lanes;
  const int seen = a.h.causal ? min(place + 1, t.len) : t.len;
  const int seen_by_all = a.h.causal ? min(q0 + 1, t.len) : t.len;
  const int seen_by_any = !live ? 0 : a.h.causal ? min(q0 + 32, t.len) : t.len;
  for (int k0 = 0, b = 0; k0 < end; k0 += kTile, b ^= 1) {
    fetched();
    __syncthreads();
    if (k0 + kTile < end) fetch(k0 + kTile, b ^ 1);
    const bool diagonal = a.h.causal && k0 >= t.r0;
    bool special = false;
    if (diagonal || k0 + kTile > t.len) special = any_special<DT, D>(s_k[b], kTile);
#pragma unroll 1
    for (int n = 0; n < 2; ++n) {
      const int k = k0 + 32 * n;
      short* ks = s_k[b] + 32 * n * D;
      const short* vs = s_v[b] + 32 * n * D;
      const TileLane<D> tl = lanes.fresh();
      s8v xp[2], xs[2];
      float* win = s_win[BIAS ? wave : 0];
      if (k < seen_by_any)
        dq_weights<DT, D, BIAS>(p, w, s_held, s_bias, win, tl, ks, vs, k, q0, seen, k + 32 > seen_by_all, xp, xs);
      if (__builtin_expect(special, 0)) {
        __syncthreads();
        clear_special<DT, D>(ks, k, t.len, diagonal, nullptr, 0);
        __syncthreads();
      }
      if (k >= seen_by_any) continue;
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
          const s8v x = tl.columns(ks, 16 * kk, d);
          w.dq[d] = mfma<DT>(x, xs[kk], w.dq[d]);
          w.pk[d] = mfma<DT>(x, xp[kk], w.pk[d]);
        }
    }
  }
  if (!live) return;
  const bool store = place < t.len;
  const float error = both_halves_sum(w.error);
  if (store && lane < 32) {
    p.a.rows[(long long)head * a.tokens + token] = w.delta + error;
    p.a.rows[(long long)(a.h.q_heads + head) * a.tokens + token] = w.z;
  }
  // dS is off by error * P, and dq by error * sum P k
  const float by = 1.f / w.c.c, off = error * (DT == EMB_F16 ? 0x1p-15f : 1.f);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) w.dq[d][i] = w.dq[d][i] * by - off * w.pk[d][i];
  // the only key that a row sees has P = 1 and dS = 0, and what the rounding of dS
  // left of dq against its correction is all that there is
  if (a.h.causal ? place == 0 : t.len == 1) {
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) w.dq[d][i] -= w.dq[d][i];  // a NaN stays one
  }
  short* dst = reinterpret_cast<short*>(const_cast<void*>(p.a.dq.p)) + token * p.a.dq.ts + head * p.a.dq.hs +
               8 * (lane >> 5);
  store_columns<DT, D>(dst, w.dq, a.h.scale, store);
}

// ---- dk, dv and dbias -----------------------------------------------------------

template <int DT, int D>
struct KeyWave {
  s8v k[D / 16], v[D / 16];
  f16v dk[D / 32], dv[D / 32];
  ColumnScale<DT> c;
};

// The second kernel's sums of the bias' gradient, a part for each wave.
template <bool BIAS>
struct GradLds {
  float sum[4][2 * EMB_MAX_BUCKETS];
};
template <>
struct GradLds<false> {};

// One step of a running sum over the neighbouring lanes of one row: adds what the
// lane that CTRL names has, if its row is the same.
template <int CTRL, int ROWS>
__device__ __forceinline__ float same_row(float v, int row) {
  const float x = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xf, false));
  const int r = __builtin_amdgcn_update_dpp(-2, row, CTRL, ROWS, 0xf, false);
  return v + (r == row ? x : 0.f);
}

// Adds a tile's dS to the sums of its rows of the bias, in a fixed order: along
// its 63 diagonals, by turning row r's lanes r places, then over the neighbouring
// diagonals of one row of the bias. `row`: of diagonal `lane`, 31 - r + c of (r, c).
__device__ __forceinline__ void add_diagonals(const f16v& s, int row, float* sum) {
  const int lane = threadIdx.x & 63, l = (lane & 31) + 4 * (lane >> 5);
  // what comes to lane l of 32 from place l + r is of diagonal 31 + l, or, from
  // behind the end, of diagonal l - 1
  float upper = 0.f, lower = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int from = l + 8 * (i / 4) + i % 4;
    const float x = __int_as_float(__builtin_amdgcn_ds_bpermute(4 * ((from & 31) | (lane & 32)), __float_as_int(s[i])));
    const bool wraps = from >= 32;
    upper += wraps ? 0.f : x;
    lower += wraps ? x : 0.f;
  }
  upper = both_halves_sum(upper);
  lower = both_halves_sum(lower);
  const float u = __shfl(upper, (lane + 1) & 31, 64), w = __shfl(lower, (lane + 1) & 31, 64);  // lanes 31 .. 62, 0 .. 30
  float v = lane < 31 ? w : u;
  if (lane == 63) {
    row = -1;
    v = 0.f;
  }
  v = same_row<0x111, 0xf>(v, row);  // one lane up, then two, four and eight inside rows of 16
  v = same_row<0x112, 0xf>(v, row);
  v = same_row<0x114, 0xf>(v, row);
  v = same_row<0x118, 0xf>(v, row);
  v = same_row<0x142, 0xa>(v, row);  // lane 15 of the row below
  v = same_row<0x143, 0xc>(v, row);  // lane 31
  const int next = __shfl_down(row, 1, 64);
  if (row >= 0 && next != row) sum[row] += v;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// From the products to P (in s, and packed) and dS (in dp): NEAR with the biases of
// each diagonal, else with `add` for all.
template <int DT, bool NEAR>
__device__ __forceinline__ void dkv_weights(float scale2, float add, const float* win, const float* zs,
                                            const float* deltas, f16v& s, f16v& dp, s8v (&x)[2]) {
  const int lane = threadIdx.x & 63, h4 = 4 * (lane >> 5);
  // diagonal of (r, c): 31 - r + c
  const float* at = win + 31 - h4 + (lane & 31);
#pragma unroll
  for (int i4 = 0; i4 < 16; i4 += 4) {
    const f4 z = *reinterpret_cast<const f4*>(zs + 2 * i4 + h4);
    const f4 delta = *reinterpret_cast<const f4*>(deltas + 2 * i4 + h4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float e = __builtin_amdgcn_exp2f(fmaf(s[i4 + j], scale2, (NEAR ? at[-(2 * i4 + j)] : add) - z[j]));
      dp[i4 + j] = e * (dp[i4 + j] - delta[j]);
      s[i4 + j] = e;
    }
  }
  pack_weights<DT>(s, x);
}

// A tile's dS into the sums of the bias' gradient.
template <bool BIAS>
__device__ __forceinline__ void add_dbias(const BackDev& p, const Biases& b, const f16v& s, GradLds<BIAS>& g,
                                          float (&far)[2]) {
  if constexpr (BIAS) {
    if (!p.a.dbias) return;
    if (b.far) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) sum += s[i];
      if (b.row < p.a.f.h.buckets.n) far[0] += sum;
      else far[1] += sum;
    } else {
      const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
      add_diagonals(s, b.row, g.sum[wave]);
    }
  }
}

// P and dS of 32 queries from q0 on, packed. edge: not all of them see every key.
template <int DT, int D, bool BIAS>
__device__ __forceinline__ void dkv_step(const BackDev& p, KeyWave<DT, D>& w, const BiasLds& sb, float* win,
                                         GradLds<BIAS>& g, float (&far)[2], const TileLane<D>& tl, const short* qs,
                                         const short* gs, const float* zs, const float* deltas, int q0, int k0, int len,
                                         bool edge, s8v (&xp)[2], s8v (&xs)[2]) {
  Biases b{};
  if (BIAS) b = biases_of(p.a.f.h, sb, q0 + 31 - k0, win);
  uint32_t bits = 0;
  if (edge) {  // none sees a key behind the end
    const int key = k0 + (threadIdx.x & 31);
    bits = row_bits(p.a.f.h.causal ? key - q0 : 0, key < len ? len - q0 : 0);
  }
  RowOps<D> qr, gr;
  qr.read(tl, qs);
  gr.read(tl, gs);
  stage();
  f16v s = qr.template times<DT>(w.k), dp = gr.template times<DT>(w.v);
  if (BIAS && !b.far) dkv_weights<DT, true>(p.scale2, 0.f, win, zs, deltas, s, dp, xp);
  else dkv_weights<DT, false>(p.scale2, b.value, win, zs, deltas, s, dp, xp);
  if (edge) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = where_bit(bits, i, s[i]);
      dp[i] = where_bit(bits, i, dp[i]);
    }
    pack_weights<DT>(s, xp);
  }
  add_dbias<BIAS>(p, b, dp, g, far);
  w.c.fit(dp, w.dk);
  pack_tile<DT>(w.c.scaled(dp), xs);
}

// 64 queries from q0 on, all of which see all keys. Products and vector work that
// do not wait for each other stand side by side: the second half's scores with the
// first half's P and dS, the first half's products with the second half's. NEAR:
// with the biases of each distance, else of the last bucket or none.
template <int DT, int D, bool BIAS, bool NEAR>
__device__ __forceinline__ void dkv_pair(const BackDev& p, KeyWave<DT, D>& w, const BiasLds& sb, float (*win)[64],
                                         GradLds<BIAS>& g, float (&far)[2], const TileLane<D>& tl, const short* qs,
                                         const short* gs, const float* zs, const float* deltas, int q0, int k0) {
  static_assert(DT == EMB_BF16, "dS goes into its product without a scale");
  RowOps<D> qr, gr;
  ColumnOps<D> gc, qc;
  qr.read(tl, qs);
  gr.read(tl, gs);
  Biases b[2] = {};
  if (BIAS) {
    b[0] = biases_of(p.a.f.h, sb, q0 + 31 - k0, win[0], NEAR);
    b[1] = biases_of(p.a.f.h, sb, q0 + 63 - k0, win[1], NEAR);
  }
  stage();
  f16v s[2], dp[2];
  s8v xp[2], xs[2][2];
  s[0] = qr.template times<DT>(w.k);
  qr.read(tl, qs + 32 * D);
  dp[0] = gr.template times<DT>(w.v);
  gr.read(tl, gs + 32 * D);
  stage();
  gc.read(tl, gs);
  s[1] = qr.template times<DT>(w.k);
  dp[1] = gr.template times<DT>(w.v);
  dkv_weights<DT, NEAR>(p.scale2, b[0].value, win[0], zs, deltas, s[0], dp[0], xp);
  interleave<D / 8, 8>();
  stage();
  qc.read(tl, qs);
  pack_tile<DT>(dp[0], xs[0]);
  gc.template times<DT>(w.dv, xp);
  gc.read(tl, gs + 32 * D);
  qc.template times<DT>(w.dk, xs[0]);
  dkv_weights<DT, NEAR>(p.scale2, b[1].value, win[1], zs + 32, deltas + 32, s[1], dp[1], xp);
  interleave<D / 8, 8>();
  stage();
  qc.read(tl, qs + 32 * D);
  pack_tile<DT>(dp[1], xs[1]);
  gc.template times<DT>(w.dv, xp);
  qc.template times<DT>(w.dk, xs[1]);
  add_dbias<BIAS>(p, b[0], dp[0], g, far);
  add_dbias<BIAS>(p, b[1], dp[1], g, far);
}

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) x += __shfl_xor(x, d, 64);
  return x;
}

// Whole tiles in pairs of half tiles, with one block a CU, or every half tile by
// itself. The gradient of 12289 items, 16 x 4 heads, with a bias: 128 wide bf16
// 1657 us in pairs and 1922 without; fp16, whose pairs would need one scale for both
// halves and with it more registers than there are, 2600 and 1705; 64 wide, where two
// blocks fit without pairs, 696 and 632 (no bias). (Each pair as measured then; now
// 1608, 1705 and 628.)
template <int DT, int D>
constexpr bool kPairs = D > 64 && DT == EMB_BF16;

// A block takes 64 keys of one key head and goes along the query tiles of 128 rows
// of each of its query heads; waves 0 and 1 take the tiles' first 64 rows for 32
// keys each, waves 2 and 3 the last 64, and are added to them at the end. So there
// are twice as many blocks, half as long, as with 128 keys.
template <int DT, int D, bool BIAS>
__global__ __launch_bounds__(256, D > 64 ? 1 : 2) void k_history_dkv(BackDev p) {
  constexpr int kPart = kRows * D;  // elements of a tile
  __shared__ __attribute__((aligned(1024))) short s_tiles[4 * kPart];  // queries twice, dout twice
  __shared__ __attribute__((aligned(16))) float s_z[2][kRows], s_delta[2][kRows];
  __shared__ BiasLds s_bias;
  __shared__ GradLds<BIAS> s_grad;
  __shared__ float s_win[BIAS ? 4 : 1][2][64];
  __shared__ Marks<D> s_marks;
  const HistoryArgs& a = p.a.f;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int kh, tile;
  head_and_tile(blockIdx.x, a.h.kv_heads, p.by_kv_heads, &kh, &tile);
  const SeqTile t = seq_tile(a, tile, kKeys);
  const bool grad = BIAS && p.a.dbias;
  float* part = p.a.part + ((long long)tile * a.h.q_heads + kh * p.m) * p.bias_rows;
  if (t.r0 >= t.len) {
    if (grad)
      for (int i = threadIdx.x; i < p.m * p.bias_rows; i += 256) part[i] = 0.f;
    return;
  }
  const int k0 = t.r0 + 32 * (wave & 1), place = k0 + (lane & 31);
  const int row0 = 64 * (wave >> 1);  // the wave's rows of a tile
  const bool live = k0 < t.len;
  const long long token = t.first + min(place, t.len - 1);
  KeyWave<DT, D> w;
  load_operands<D>(a.k, token, kh, w.k);
  load_operands<D>(a.v, token, kh, w.v);
#pragma unroll
  for (int d = 0; d < D / 32; ++d) w.dk[d] = w.dv[d] = f16v{};
  const int begin = a.h.causal ? t.r0 / kRows * kRows : 0;
  const uint32_t q_step = 2 * (uint32_t)a.q.ts, g_step = 2 * (uint32_t)p.a.dout.ts;
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_elem*)s_tiles;
  const uint32_t lds_z = (uint32_t)(uintptr_t)(lds_word*)&s_z[0][0];
  const uint32_t lds_delta = (uint32_t)(uintptr_t)(lds_word*)&s_delta[0][0];
  const RowFetch<D> f;
  const TileLane<D> lanes;
  bool marked = false;
  s_marks.clear();
  if (BIAS) stage_bounds(a.h, s_bias);
  for (int hh = 0; hh < p.m; ++hh) {
    const int head = kh * p.m + hh;
    const uint64_t q_at = uniform((uint64_t)a.q.p + 2 * (t.first * a.q.ts + head * a.q.hs));
    const uint64_t g_at = uniform((uint64_t)p.a.dout.p + 2 * (t.first * p.a.dout.ts + head * p.a.dout.hs));
    // the rows' sums and z: waves 0 and 2 fetch the one, 1 and 3 the other
    const uint64_t word_at = uniform(
        (uint64_t)(p.a.rows + (long long)((wave & 1 ? a.h.q_heads : 0) + head) * a.tokens + t.first));
    auto fetch = [&](int q0, int b) {
      const int last = t.len - 1 - q0;
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        f.rows(q_at + (uint64_t)q0 * q_step, q_step, 64 * n, last, lds + 2 * (b * kPart + n * 64 * D));
        f.rows(g_at + (uint64_t)q0 * g_step, g_step, 64 * n, last, lds + 2 * ((2 + b) * kPart + n * 64 * D));
      }
      fetch_word_to_lds(word_at + 4 * (uint64_t)q0, 4 * (uint32_t)min(row0 + lane, last),
                        (wave & 1 ? lds_z : lds_delta) + 4 * (b * kRows + row0));
    };
    __syncthreads();  // the last head's tiles and bias are done with
    fetch(begin, 0);
    if (BIAS) stage_bias(a, head, s_bias);
    if constexpr (BIAS) {
      for (int i = threadIdx.x; i < 4 * 2 * EMB_MAX_BUCKETS; i += 256) (&s_grad.sum[0][0])[i] = 0.f;
    }
    float far[2] = {0.f, 0.f};
    for (int q0 = begin, b = 0; q0 < t.len; q0 += kRows, b ^= 1) {
      fetched();
      __syncthreads();
      if (q0 + kRows < t.len) fetch(q0 + kRows, b ^ 1);
      short *qs = s_tiles + b * kPart, *gs = s_tiles + (2 + b) * kPart;
      const bool diagonal = a.h.causal && q0 < t.r0 + kKeys;
      bool special = false;
      if (diagonal || q0 + kRows > t.len)
        special = any_special<DT, D>(qs, kRows) + any_special<DT, D>(gs, kRows) > 0;  // each has its barrier
      marked |= special;
      float(*wins)[64] = s_win[BIAS ? wave : 0];
      if constexpr (kPairs<DT, D>) {
        if (__builtin_expect(!special && live && q0 + row0 + 64 <= t.len &&
                                 (a.h.causal ? q0 + row0 >= k0 + 31 : k0 + 32 <= t.len), 1)) {
          const int q = q0 + row0;
          const short *q_rows = qs + row0 * D, *g_rows = gs + row0 * D;
          const float *zs = s_z[b] + row0, *deltas = s_delta[b] + row0;
          if (BIAS && !all_far(a.h, q + 63 - k0, q - 31 - k0))
            dkv_pair<DT, D, BIAS, BIAS>(p, w, s_bias, wins, s_grad, far, lanes.fresh(), q_rows, g_rows, zs, deltas, q, k0);
          else
            dkv_pair<DT, D, BIAS, false>(p, w, s_bias, wins, s_grad, far, lanes.fresh(), q_rows, g_rows, zs, deltas, q, k0);
          continue;
        }
      }
      float* win = wins[0];
#pragma unroll 1
      for (int n = 0; n < 2; ++n) {
        const int r = row0 + 32 * n, q = q0 + r;
        const TileLane<D> tl = lanes.fresh();
        s8v xp[2], xs[2];
        const bool some = live && q < t.len && !(a.h.causal && q + 31 < k0);
        const float *zs = s_z[b] + r, *deltas = s_delta[b] + r;
        if (some)
          dkv_step<DT, D, BIAS>(p, w, s_bias, win, s_grad, far, tl, qs + r * D, gs + r * D, zs, deltas, q, k0,
                                t.len, q + 32 > t.len || (a.h.causal ? q < k0 + 31 : k0 + 32 > t.len), xp, xs);
        if (__builtin_expect(special, 0)) {
          __syncthreads();
          for (int half = 0; half < 2; ++half) {
            const int at = 64 * half + 32 * n;
            clear_special<DT, D>(qs + at * D, q0 + at, t.len, diagonal, (Marks<D>*)nullptr, 0);
            clear_special<DT, D>(gs + at * D, q0 + at, t.len, diagonal, &s_marks, -1);
          }
          __syncthreads();
        }
        if (!some) continue;
        add_product<DT, D>(w.dv, tl, gs + r * D, xp);
        add_product<DT, D>(w.dk, tl, qs + r * D, xs);
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
  // waves 2 and 3 hand theirs to 0 and 1
  float* hand = reinterpret_cast<float*>(s_tiles) + (wave & 1) * 64 * D + lane;
  const float by = 1.f / w.c.c;
  __syncthreads();
  if (wave >= 2) {
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        hand[64 * (16 * d + i)] = w.dk[d][i] * by;
        hand[64 * (16 * (D / 32 + d) + i)] = w.dv[d][i];
      }
  }
  __syncthreads();
  if (wave >= 2 || !live) return;
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      w.dk[d][i] = w.dk[d][i] * by + hand[64 * (16 * d + i)];
      w.dv[d][i] += hand[64 * (16 * (D / 32 + d) + i)];
    }
  if (__builtin_expect(marked, 0)) add_marks<D>(w.dv, s_marks, -place);
  const bool store = place < t.len;
  short* dk = reinterpret_cast<short*>(const_cast<void*>(p.a.dk.p)) + token * p.a.dk.ts + kh * p.a.dk.hs + 8 * (lane >> 5);
  short* dv = reinterpret_cast<short*>(const_cast<void*>(p.a.dv.p)) + token * p.a.dv.ts + kh * p.a.dv.hs + 8 * (lane >> 5);
  store_columns<DT, D>(dk, w.dk, a.h.scale, store);
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
  if (p.a.f.tokens > 0) {
    k_history_dq<DT, D, BIAS><<<(unsigned)(p.q_tiles * h.q_heads), 256, 0, st>>>(p);
    if (hipError_t e = hipGetLastError()) return e;
    k_history_dkv<DT, D, BIAS><<<(unsigned)(p.k_tiles * h.kv_heads), 256, 0, st>>>(p);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (BIAS && p.a.dbias)
    k_history_dbias<<<(unsigned)(p.bias_rows * h.q_heads), 256, 0, st>>>(p.a.part, p.a.f.tokens > 0 ? p.k_tiles : 0,
                                                                        h.q_heads, p.bias_rows, p.a.dbias);
  return hipGetLastError();
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
  p.part_off = ((size_t)tokens * h.q_heads * 8 + 255) & ~size_t(255);
  p.bytes = p.part_off + (size_t)(seq_tiles(tokens, seqs, kKeys) * h.q_heads * rows * 4);
  return p;
}

hipError_t launch_history_back(const HistoryBackArgs& a, hipStream_t st) {
  BackDev p{};
  p.a = a;
  p.scale2 = a.f.h.scale * kLog2e;
  p.m = a.f.h.q_heads / a.f.h.kv_heads;
  p.by_m = fast_div((uint32_t)p.m);
  p.by_heads = fast_div((uint32_t)a.f.h.q_heads);
  p.by_kv_heads = fast_div((uint32_t)a.f.h.kv_heads);
  p.q_tiles = (int)seq_tiles(a.f.tokens, a.f.seqs, kRows);
  p.k_tiles = (int)seq_tiles(a.f.tokens, a.f.seqs, kKeys);
  p.bias_rows = a.f.h.buckets.n * (a.f.h.causal ? 1 : 2);
  return a.f.h.dtype == EMB_BF16 ? launch_t<EMB_BF16>(p, st) : launch_t<EMB_F16>(p, st);
}

}  // namespace emb
