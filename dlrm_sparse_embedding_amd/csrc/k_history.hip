// Attention of a ragged batch of histories over themselves, with a learned bias
// by relative position.
//
// Mathematics. For the query at place i of a history and the keys j it sees,
//     s_j = log2(e) (scale q.k_j + bias[row(i - j)]),  out = sum_j 2^(s_j - z) v_j,
//     z = log2 sum_j 2^(s_j),
// in one pass over the keys with a running maximum. The bias of a tile of
// 32 x 32 is worked out once for its 63 diagonals, one a lane, not for each pair;
// beyond the last bucket's start it is one number.
//
// Layout. A block takes 128 queries of one head, each wave 32; tiles of 64 keys
// and values go through LDS for all of them, the next ones on their way while
// these are worked on. S^T = K Q^T: a lane holds 32 keys' scores of ONE query,
// and its probabilities already lie as the operand of O^T = V^T P^T.
//
// Bound by the products and the vector work of a wave, which overlap with another
// wave's only in part: 12289 items, 16 x 4 heads of 128, causal, 267 us without a
// bias (870 TFLOP/s), 306 with one of 64 buckets up to 1024, where a third of the
// tiles have a bias for each diagonal, which each wave works out for itself (297
// with the biases of all near distances in a table, not taken up); heads of 64
// 164 us (714 TFLOP/s: as many exponentials for half the products). Waits that the compiler puts into the loop
// (operands not there before it, spilled registers) also wait for the next tile's
// transfer: without them the long cases went from 1137 to 1090 us.
//
// Precision. Scores, maxima, sums and outputs are fp32; probabilities are rounded
// to the heads' type for the product with V (half a step: 2^-8 relative for
// bf16, 2^-11 for fp16), scaled by 2^8 so that fp16 keeps its full precision
// down to 2^-22 of a row's largest. The sum that divides is of the unrounded ones.
#include <algorithm>

#include "history_device.h"

namespace emb {

namespace {

constexpr float kShift = 8.f;  // probabilities carry this many powers of two
constexpr float kSlack = 7.f;  // and this many more before the reference moves
constexpr int kRows = 128;     // queries of a block

template <int DT, int D>
struct Wave {
  s8v q[D / 16];
  f16v o[D / 32];
  float mx, sum;  // running maximum (log2 units) and the lane's part of the sum
};

// Probabilities of 32 keys, packed. edge: not every row sees all of them.
template <int DT, int D, bool BIAS>
__device__ __forceinline__ void weights_of(const HistoryArgs& a, float scale2, Wave<DT, D>& w, const BiasLds& sb,
                                           float* win, const TileLane<D>& tl, const short* ks, int k0, int q0, int seen, bool edge,
                                           s8v (&p)[2]) {
  const int lane = threadIdx.x & 63;
  Biases b{};
  if (BIAS) b = biases_of(a.h, sb, q0 + 31 - k0, win);
  f16v s[1];
  s[0] = f16v{};
#pragma unroll
  for (int i = 0; i < D / 16; ++i) s[0] = mfma<DT>(tl.rows(ks, 0, i), w.q[i], s[0]);
  float mul = scale2, add = 0.f;  // a score is s * mul + add
  if (BIAS && b.far) add = b.value;
  if (BIAS && !b.far) {
    const float* at = win + 4 * (lane >> 5) + 31 - (lane & 31);
#pragma unroll
    for (int i = 0; i < 16; ++i) s[0][i] = fmaf(s[0][i], scale2, at[8 * (i / 4) + i % 4]);
    mul = 1.f;
  }
  if (edge) mask_tile(s[0], k0, seen);
  const float top = fmaf(both_halves_max(top_of(s)), mul, add);
  const bool up = top > w.mx + kSlack;
  if (__ballot(up)) {
    const float keep = up ? __builtin_amdgcn_exp2f(w.mx - top) : 1.f;
    w.mx = up ? top : w.mx;
    w.sum *= keep;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) w.o[d][i] *= keep;
  }
  add += kShift - (w.mx == kNegInf ? 0.f : w.mx);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    s[0][i] = __builtin_amdgcn_exp2f(fmaf(s[0][i], mul, add));
    sum += s[0][i];
  }
  w.sum += sum;
  pack_tile<DT>(s[0], p);
}

template <int DT, int D, bool BIAS>
__global__ __launch_bounds__(256, 2) void k_history(HistoryArgs a, int tiles, FastDiv by_heads, FastDiv by_m) {
  __shared__ __attribute__((aligned(1024))) short s_k[2][kTile * D], s_v[2][kTile * D];
  __shared__ BiasLds s_bias;
  __shared__ float s_win[BIAS ? 4 : 1][64];
  __shared__ Marks<D> s_marks;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  report_offsets(a.offsets, a.seqs, a.tokens, a.h.error);
  int head, tile;
  head_and_tile(blockIdx.x, a.h.q_heads, by_heads, &head, &tile);
  const SeqTile t = seq_tile(a, tiles - 1 - tile, kRows);  // later tiles, which see more, first
  if (t.r0 >= t.len) return;
  const int kh = div_by(by_m, head);
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
  s_marks.clear();
  const int q0 = t.r0 + 32 * wave, place = q0 + (lane & 31);
  const bool live = q0 < t.len;
  const long long token = t.first + min(place, t.len - 1);
  Wave<DT, D> w;
  load_operands<D>(a.q, token, head, w.q);
#pragma unroll
  for (int d = 0; d < D / 32; ++d) w.o[d] = f16v{};
  w.mx = kNegInf;
  w.sum = 0.f;
  const int seen = a.h.causal ? min(place + 1, t.len) : t.len;
  const int seen_by_all = a.h.causal ? min(q0 + 1, t.len) : t.len;
  const int seen_by_any = !live ? 0 : a.h.causal ? min(q0 + 32, t.len) : t.len;
  const float scale2 = a.h.scale * kLog2e;
  const TileLane<D> lanes;
  bool marked = false;
  for (int k0 = 0, b = 0; k0 < end; k0 += kTile, b ^= 1) {
    fetched();
    __syncthreads();
    if (k0 + kTile < end) fetch(k0 + kTile, b ^ 1);
    const bool diagonal = a.h.causal && k0 >= t.r0;
    bool special = false;
    if (diagonal || k0 + kTile > t.len) special = any_special<DT, D>(s_v[b], kTile);
    marked |= special;
#pragma unroll 1
    for (int n = 0; n < 2; ++n) {
      const int k = k0 + 32 * n;
      short* vs = s_v[b] + 32 * n * D;
      const TileLane<D> tl = lanes.fresh();
      s8v p[2];
      float* win = s_win[BIAS ? wave : 0];
      const bool some = k < seen_by_any;
      if (some)
        weights_of<DT, D, BIAS>(a, scale2, w, s_bias, win, tl, s_k[b] + 32 * n * D, k, q0, seen, k + 32 > seen_by_all, p);
      if (__builtin_expect(special, 0)) {
        clear_special<DT, D>(vs, k, t.len, diagonal, &s_marks, 1);
        __syncthreads();
      }
      if (some) add_product<DT, D>(w.o, tl, vs, p);
    }
  }
  if (!live) return;
  const float total = both_halves_sum(w.sum);
  const bool some = !(total == 0.f);  // a NaN counts
  const float inv = some ? 1.f / total : 0.f;
  const bool store = place < t.len;
  if (a.lse && store && lane < 32)
    a.lse[token * a.h.q_heads + head] = some ? (w.mx - kShift + __log2f(total)) * kLn2 : kNegInf;
  if (!some) {
#pragma unroll
    for (int d = 0; d < D / 32; ++d) w.o[d] = f16v{};
  }
  if (__builtin_expect(marked, 0) && some) add_marks<D>(w.o, s_marks, place);
  short* dst = reinterpret_cast<short*>(const_cast<void*>(a.out.p)) + token * a.out.ts + head * a.out.hs + 8 * (lane >> 5);
  store_columns<DT, D>(dst, w.o, inv, store);
}

template <int DT, int D>
hipError_t launch(const HistoryArgs& a, hipStream_t st) {
  const long long tiles = seq_tiles(a.tokens, a.seqs, kRows);
  const unsigned blocks = (unsigned)(tiles * a.h.q_heads);
  const FastDiv by_heads = fast_div((uint32_t)a.h.q_heads);
  const FastDiv by_m = fast_div((uint32_t)(a.h.q_heads / a.h.kv_heads));
  if (a.bias) k_history<DT, D, true><<<blocks, 256, 0, st>>>(a, (int)tiles, by_heads, by_m);
  else k_history<DT, D, false><<<blocks, 256, 0, st>>>(a, (int)tiles, by_heads, by_m);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_history(const HistoryArgs& a, hipStream_t st) {
  const bool bf = a.h.dtype == EMB_BF16;
  switch (a.h.dim) {
    case 64: return bf ? launch<EMB_BF16, 64>(a, st) : launch<EMB_F16, 64>(a, st);
    case 96: return bf ? launch<EMB_BF16, 96>(a, st) : launch<EMB_F16, 96>(a, st);
    default: return bf ? launch<EMB_BF16, 128>(a, st) : launch<EMB_F16, 128>(a, st);
  }
}

}  // namespace emb
