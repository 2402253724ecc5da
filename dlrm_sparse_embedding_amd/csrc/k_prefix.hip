// Attention of many queries over a prefix that their group shares and over
// their own sequence, both in a paged cache.
//
// Mathematics. For one query row q and the slots it sees,
//     out = sum_j 2^(s_j - z) v_j,  z = log2 sum_j 2^(s_j),  s_j = log2(e) scale q.k_j,
// in one pass with a running maximum: a part of the slots gives a partial
// output and its z, and parts are joined with the weights 2^(z_i - max z). So
// the prefix is read once for all queries of its group, whatever their
// number, and long slot ranges are split over the chip.
//
// Layout. A tile is 32 slots by 32 query rows of one cache head (a row is a
// query token and one of the m query heads that read the cache head). The
// product is taken transposed, S^T = K Q^T, with the 32x32x16 matrix
// instruction: a lane then holds 16 slots of ONE query row (its column, lane %
// 32; the other 16 are in lane + 32), so the softmax needs one exchange
// between lanes, and its probabilities already lie as the B operand of O^T =
// V^T P^T: contraction index 8 h + j (h = lane / 32) stands for slot 8 (j / 4)
// + 4 h + j % 4 on both sides. V's side of it, 4 consecutive slots of one
// column, is what the transposed LDS read returns.
//
// Precision. Scores, maxima, sums and outputs are fp32. The probabilities are
// rounded to the cache's type for the product with V (at most 2^-8 relative for
// bf16 and 2^-11 for fp16, half a step; the sum that divides them is of
// the unrounded ones). They are scaled by 2^8, so that fp16 keeps its full
// precision down to 2^-22 of a row's largest.
#include <algorithm>
#include <cmath>

#include "emb_device.h"
#include "seq_internal.h"

namespace emb {

namespace {

typedef short s4v __attribute__((ext_vector_type(4)));
typedef short s8v __attribute__((ext_vector_type(8)));
typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
typedef _Float16 hf8 __attribute__((ext_vector_type(8)));
typedef _Float16 hf2 __attribute__((ext_vector_type(2)));
typedef float fl2 __attribute__((ext_vector_type(2)));
typedef float f16v __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) s4v lds_s4v;

constexpr float kShift = 8.f;  // probabilities carry this many powers of two
constexpr float kSlack = 7.f;  // and this many more before the reference moves
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

struct PrefixDev {
  PrefixArgs a;
  float scale2;  // |scale| * log2(e), never 0
  uint32_t q_sign;  // sign bits of two elements where the scale is negative
  int m;         // query heads of a cache head
  FastDiv by_m;
  int nps, nos;
  int prefix_blocks, prefix_tiles;  // tiles: upper bound, blocks = tiles * heads * nps
  int own_tiles, own_tq;            // tiles of own_tq tokens each: upper bound
  float* part_o;
  float* part_lse;
};

__device__ __forceinline__ int div_by(const FastDiv d, int n) {
  return (int)(((uint64_t)(uint32_t)n * d.mul) >> d.shift);
}

__device__ __forceinline__ void flag(const PrefixDev& p, int bit) {
  if (p.a.kv.error) atomicOr(p.a.kv.error, bit);
}

// First token of sequence b (b <= seqs), kept inside the tokens.
__device__ __forceinline__ int first_token(const PrefixDev& p, int b) {
  const int t = p.a.offsets ? p.a.offsets[b] : b;
  return min(max(t, 0), p.a.tokens);
}

// First token of group g (g <= groups).
__device__ __forceinline__ int group_token(const PrefixDev& p, int g) {
  const int b = p.a.group_offsets[g];
  return first_token(p, min(max(b, 0), p.a.seqs));
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

// What one wave works on: 32 rows of cache head `h` and the slots [k0, k1) of
// a page table row.
struct Rows {
  int t0;    // first token
  int r0;    // first row, counted from t0 * m
  int rows;  // rows of the item, counted from t0 * m
  int h;
};

// The wave's state for its 32 rows, one row per lane column.
template <int DT, int D>
struct Wave {
  s8v q[D / 16];
  f16v o[D / 32];
  float mx;   // running maximum of the scores (log2 units)
  float sum;  // this lane's part of the sum
};

template <int DT, int D>
__device__ __forceinline__ void load_q(const PrefixDev& p, const Rows& it, Wave<DT, D>& w) {
  const int lane = threadIdx.x & 63;
  const int row = it.r0 + (lane & 31);
  const int rr = min(row, it.rows - 1);  // rows past the end repeat the last one; they are not stored
  const int j = div_by(p.by_m, rr);
  const int head = it.h * p.m + rr - j * p.m;
  const short* src = reinterpret_cast<const short*>(p.a.q.p) + (long long)(it.t0 + j) * p.a.q.ts + head * p.a.q.hs;
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    u4 x = *reinterpret_cast<const u4*>(src + 16 * s + 8 * (lane >> 5));
    x ^= p.q_sign;  // a negative scale is taken into q, so that maxima stay maxima
    w.q[s] = __builtin_bit_cast(s8v, x);
  }
#pragma unroll
  for (int d = 0; d < D / 32; ++d) w.o[d] = f16v{};
  w.mx = kNegInf;
  w.sum = 0.f;
}

// Row (page, slot) of a slot's keys and values; a slot without a page reads
// page 0 and raises the flag (its values are then meaningless, but in range).
__device__ __forceinline__ void locate(const PrefixDev& p, const int* pages, int slot, int* page, int* in_page) {
  const int col = div_by(p.a.kv.by_page, slot);
  int pg = pages[col];
  if (pg < 0 || pg >= p.a.kv.pages) {
    flag(p, kKvBadPage);
    pg = 0;
  }
  *page = pg;
  *in_page = slot - col * p.a.kv.page;
}

// Elements between rows of a wave's own V tile: 4 rows, 64 bytes of each, are
// read at once and have to lie in different banks of the 64.
template <int D>
constexpr int v_pad() {
  return D == 96 ? 0 : 32;
}

// One wave's V tile: 32 slots.
template <int D>
constexpr int v_tile_elems() {
  return 32 * (D + v_pad<D>());
}

// V^T operand of 16 slots from slot base `kk` and 32 columns from d0.
template <int D>
__device__ __forceinline__ s8v read_vt(const short* v, int kk, int d0) {
  const int lane = threadIdx.x & 63;
  const int q = lane & 15;
  const short* at = v + (kk + 4 * (lane >> 5) + (q >> 2)) * (D + v_pad<D>()) + d0 + 16 * ((lane >> 4) & 1) + 4 * (q & 3);
  const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)at);
  const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(at + 8 * (D + v_pad<D>())));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
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

// Takes N tiles' scores (raw products) into the running maximum. The outputs
// are rescaled only where a maximum has grown by more than kSlack since the
// reference was set: any reference gives the same quotient, and the slack
// keeps the probabilities below 2^15.
template <int DT, int D, int N>
__device__ __forceinline__ void refer(const PrefixDev& p, Wave<DT, D>& w, const f16v (&s)[N]) {
  const float top = both_halves_max(top_of(s)) * p.scale2;
  if (__ballot(top > w.mx + kSlack)) {
    const float mx = fmaxf(w.mx, top);
    const float keep = mx == kNegInf ? 1.f : __builtin_amdgcn_exp2f(w.mx - mx);
    w.mx = mx;
    w.sum *= keep;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) w.o[d][i] *= keep;
  }
}

// Probabilities of N tiles of 32 slots, packed for the V product, and their
// sum. Masked scores are -infinity already.
template <int DT, int D, int N>
__device__ __forceinline__ void probabilities(const PrefixDev& p, Wave<DT, D>& w, f16v (&s)[N], s8v (&prob)[2 * N]) {
  const float add = kShift - (w.mx == kNegInf ? 0.f : w.mx);
  float sum = 0.f;
#pragma unroll
  for (int k = 0; k < 2 * N; ++k) {
    f16v& x = s[k / 2];
    const int i0 = 8 * (k % 2);
#pragma unroll
    for (int i = i0; i < i0 + 8; ++i) {
      x[i] = __builtin_amdgcn_exp2f(fmaf(x[i], p.scale2, add));
      sum += x[i];
    }
    u4 b;
    b.x = pack2<DT>(x[i0], x[i0 + 1]);
    b.y = pack2<DT>(x[i0 + 2], x[i0 + 3]);
    b.z = pack2<DT>(x[i0 + 4], x[i0 + 5]);
    b.w = pack2<DT>(x[i0 + 6], x[i0 + 7]);
    prob[k] = __builtin_bit_cast(s8v, b);
  }
  w.sum += sum;
}

// Clears the scores of a tile's slots at and beyond `seen` (the lane's own limit).
__device__ __forceinline__ void mask_tile(f16v& s, int slot0, int seen) {
  const int h4 = 4 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (slot0 + 8 * (i / 4) + h4 + i % 4 >= seen) s[i] = kNegInf;
}

// One wave over slots k0, k0 + step, .. below k1 in tiles of 32, the keys
// straight into registers (each is used once) and the values through the
// wave's own LDS tile. `seen` is the lane's limit, lim_lo and lim_hi the
// smallest and largest of the wave's; no slot at or beyond lim_hi is read.
// `token` tells rows of unlike limits apart.
template <int DT, int D>
__device__ void wave_slots(const PrefixDev& p, Wave<DT, D>& w, const int* pages, int h, int k0, int k1, int step,
                           int seen, int lim_lo, int lim_hi, short* v) {
  const int lane = threadIdx.x & 63;
  const KvView& kv = p.a.kv;
  constexpr int VL = 32 * D / 8 / 64;  // 16-byte pieces of a V tile for each lane
  k1 = min(k1, lim_hi);
  for (int k = k0; k < k1; k += step) {
    int page, in_page;
    // slots past the end read the last one again; their scores are masked
    locate(p, pages, min(k + (lane & 31), lim_hi - 1), &page, &in_page);
    const short* kp = reinterpret_cast<const short*>(kv.k) + page * kv.kps + in_page * kv.kss + h * kv.khs;
    s8v kf[D / 16];
#pragma unroll
    for (int s = 0; s < D / 16; ++s) kf[s] = *reinterpret_cast<const s8v*>(kp + 16 * s + 8 * (lane >> 5));
    s8v vr[VL];
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int piece = i * 64 + lane, row = piece / (D / 8);
      const int pg = __shfl(page, row, 64), sl = __shfl(in_page, row, 64);
      vr[i] = *reinterpret_cast<const s8v*>(reinterpret_cast<const short*>(kv.v) + pg * kv.vps + sl * kv.vss +
                                            h * kv.vhs + 8 * (piece % (D / 8)));
    }
    f16v s[1] = {};
#pragma unroll
    for (int i = 0; i < D / 16; ++i) s[0] = mfma<DT>(kf[i], w.q[i], s[0]);
#pragma unroll
    for (int i = 0; i < VL; ++i) {
      const int piece = i * 64 + lane;
      *reinterpret_cast<s8v*>(v + piece / (D / 8) * (D + v_pad<D>()) + 8 * (piece % (D / 8))) = vr[i];
    }
    s8v prob[2];
    if (k + 32 > lim_lo) mask_tile(s[0], k, seen);
    refer<DT, D, 1>(p, w, s);
    probabilities<DT, D, 1>(p, w, s, prob);
    if (k + 32 <= lim_lo || lim_lo == lim_hi) {
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) w.o[d] = mfma<DT>(read_vt<D>(v, 16 * kk, 32 * d), prob[kk], w.o[d]);
    } else {
      // Rows of unlike limits in one tile: a zero probability must not meet a
      // value that its row does not see (0 * infinity). One product for each
      // limit, the values beyond it cleared, and each row keeps its own.
      for (int lim = lim_hi; lim >= lim_lo; --lim) {
        if (!__ballot(seen == lim)) continue;
        for (int i = lane; i < 32 * (D / 8); i += 64) {
          const int row = i / (D / 8);
          if (k + row >= lim) *reinterpret_cast<s8v*>(v + row * (D + v_pad<D>()) + 8 * (i % (D / 8))) = s8v{};
        }
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
          f16v o = {};
#pragma unroll
          for (int kk = 0; kk < 2; ++kk) o = mfma<DT>(read_vt<D>(v, 16 * kk, 32 * d), prob[kk], o);
          if (seen == lim) {
#pragma unroll
            for (int i = 0; i < 16; ++i) w.o[d][i] += o[i];
          }
        }
      }
    }
  }
}

// Stores the wave's rows as partial output `part`.
template <int DT, int D>
__device__ __forceinline__ void store_part(const PrefixDev& p, const Rows& it, Wave<DT, D>& w, int part) {
  const int lane = threadIdx.x & 63;
  const int row = it.r0 + (lane & 31);
  const float total = both_halves_sum(w.sum);
  if (row >= it.rows) return;
  const int j = div_by(p.by_m, row);
  const int head = it.h * p.m + row - j * p.m;
  const long long at = ((long long)part * p.a.tokens + it.t0 + j) * p.a.q_heads + head;
  const bool some = !(total == 0.f);  // a NaN counts
  if (lane < 32) p.part_lse[at] = some ? w.mx - kShift + __log2f(total) : kNegInf;
  if (!some) return;
  const float inv = 1.f / total;
  float* dst = p.part_o + at * D + 4 * (lane >> 5);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<f4*>(dst + 32 * d + 8 * i) =
          f4{w.o[d][4 * i] * inv, w.o[d][4 * i + 1] * inv, w.o[d][4 * i + 2] * inv, w.o[d][4 * i + 3] * inv};
}

// A prefix block's work: tile `tile` of the groups' tiles of `rows` rows, and a
// part of the prefix. False where there is none.
struct PrefixItem {
  Rows it;
  const int* pages;
  int k0, k1;
};
__device__ __forceinline__ bool prefix_item(const PrefixDev& p, int id, int rows, PrefixItem* w, int* part) {
  // the tile fastest (neighbours read the same slots), then the part, then the cache head
  const int tile = id % p.prefix_tiles;
  id /= p.prefix_tiles;
  *part = id % p.nps;
  const int h = id / p.nps;
  if (h >= p.a.kv.heads) return false;  // the grid is a multiple of 8
  // tile i of the group whose tiles start at g + (its first row) / rows
  const int g = wave_find(p.a.groups, tile, [&](int i) { return i + group_token(p, i) * p.m / rows; });
  const int t0 = group_token(p, g), t1 = group_token(p, g + 1);
  w->it = Rows{t0, (tile - (g + t0 * p.m / rows)) * rows, (t1 - t0) * p.m, h};
  if (tile == 0 && *part == 0 && h == 0 && threadIdx.x == 0 &&
      (p.a.group_offsets[0] != 0 || p.a.group_offsets[p.a.groups] != p.a.seqs))
    flag(p, kKvBadOffsets);
  if (w->it.r0 < 0 || w->it.r0 >= w->it.rows) return false;  // the bound counts more tiles than there are
  int len = p.a.prefix_lens[g];
  const long long cap = (long long)p.a.pwidth * p.a.kv.page;
  if (len < 0 || len > cap) {
    if (threadIdx.x == 0) flag(p, kKvBadPage);
    len = len < 0 ? 0 : (int)cap;
  }
  const int chunk = max(256, ((len + p.nps - 1) / p.nps + 127) & ~127);
  w->k0 = (int)min((long long)*part * chunk, (long long)len);
  w->k1 = min(w->k0 + chunk, len);
  w->pages = p.a.prefix_table + (long long)g * p.a.pwidth;
  return true;
}

// Own sequences: each wave of block `block` for itself takes a tile of rows, a
// cache head and a part of the sequence; part fastest, then the tile, then the
// cache head.
template <int DT, int D>
__device__ void own_part(const PrefixDev& p, int block, short* v) {
  const int lane = threadIdx.x & 63;
  int id = block * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = id % p.nos;
  id /= p.nos;
  const int tile = id % p.own_tiles;
  const int h = id / p.own_tiles;
  if (h >= p.a.kv.heads) return;
  const int b = wave_find(p.a.seqs, tile, [&](int i) { return i + first_token(p, i) / p.own_tq; });
  const int t0 = first_token(p, b), t1 = first_token(p, b + 1);
  const int j0 = (tile - (b + t0 / p.own_tq)) * p.own_tq;  // first token of the tile, counted from t0
  if (tile == 0 && part == 0 && h == 0 && lane == 0 && p.a.offsets &&
      (p.a.offsets[0] != 0 || p.a.offsets[p.a.seqs] != p.a.tokens))
    flag(p, kKvBadOffsets);
  const int n = t1 - t0;
  if (j0 < 0 || j0 >= n) return;
  int len = p.a.lens[b];
  const long long cap = (long long)p.a.width * p.a.kv.page;
  if (len < 0 || len > cap) {
    if (lane == 0) flag(p, kKvBadPage);
    len = len < 0 ? 0 : (int)cap;
  }
  const int j1 = min(j0 + p.own_tq, n);
  const int lim_lo = max(len - n + j0 + 1, 0), lim_hi = max(len - n + j1, 0);
  const int chunk = max(128, ((lim_hi + p.nos - 1) / p.nos + 31) & ~31);
  const int k0 = part * chunk;
  // more than 32 query heads of one cache head: a token takes several tiles of rows
  for (int r0 = j0 * p.m; r0 < j1 * p.m; r0 += 32) {
    const Rows it{t0, r0, j1 * p.m, h};
    Wave<DT, D> w;
    load_q<DT, D>(p, it, w);
    const int j = div_by(p.by_m, min(r0 + (lane & 31), it.rows - 1));
    const int seen = max(len - n + j + 1, 0);
    if (k0 < lim_hi)
      wave_slots<DT, D>(p, w, p.a.table + (long long)b * p.a.width, h, k0, min(k0 + chunk, lim_hi), 32, seen, lim_lo,
                        lim_hi, v);
    store_part<DT, D>(p, it, w, p.nps + part);
  }
}

// Few rows: a block takes one tile of 32 rows, a cache head and a part of the
// prefix; its four waves take every fourth tile of slots and are joined in LDS.
template <int DT, int D>
__global__ __launch_bounds__(256, 2) void k_attend(PrefixDev p) {
  constexpr int OS = D + 4;  // row stride of the joined outputs (floats): rows start 4 banks apart
  constexpr size_t kV = 4 * v_tile_elems<D>() * sizeof(short), kO = (2 * 32 * OS + 4 * 64) * sizeof(float);
  __shared__ __attribute__((aligned(16))) char smem[kV > kO ? kV : kO];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  short* v = reinterpret_cast<short*>(smem) + wave * v_tile_elems<D>();
  Wave<DT, D> w;
  if ((int)blockIdx.x < p.prefix_blocks) {
    PrefixItem x;
    int part;
    if (!prefix_item(p, blockIdx.x, 32, &x, &part)) return;
    const Rows it = x.it;
    load_q<DT, D>(p, it, w);
    wave_slots<DT, D>(p, w, x.pages, it.h, x.k0 + 32 * wave, x.k1, 128, x.k1, x.k1, x.k1, v);
    // join: waves 2 and 3 into 0 and 1, then 1 into 0
    float* so = reinterpret_cast<float*>(smem);
    float* sm = so + 2 * 32 * OS;
    for (int half = 2; half >= 1; half >>= 1) {
      __syncthreads();
      if (wave >= half && wave < 2 * half) {
        float* dst = so + (wave - half) * 32 * OS + (lane & 31) * OS + 4 * (lane >> 5);
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f4*>(dst + 32 * d + 8 * i) =
                f4{w.o[d][4 * i], w.o[d][4 * i + 1], w.o[d][4 * i + 2], w.o[d][4 * i + 3]};
        sm[(wave - half) * 128 + lane] = w.mx;
        sm[(wave - half) * 128 + 64 + lane] = w.sum;
      }
      __syncthreads();
      if (wave < half) {
        const float omx = sm[wave * 128 + lane], osum = sm[wave * 128 + 64 + lane];
        const float mx = fmaxf(w.mx, omx);
        const float ka = mx == kNegInf ? 1.f : __builtin_amdgcn_exp2f(w.mx - mx);
        const float kb = mx == kNegInf ? 0.f : __builtin_amdgcn_exp2f(omx - mx);
        w.mx = mx;
        w.sum = w.sum * ka + osum * kb;
        const float* src = so + wave * 32 * OS + (lane & 31) * OS + 4 * (lane >> 5);
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f4 x = *reinterpret_cast<const f4*>(src + 32 * d + 8 * i);
#pragma unroll
            for (int c = 0; c < 4; ++c) w.o[d][4 * i + c] = w.o[d][4 * i + c] * ka + x[c] * kb;
          }
      }
    }
    if (wave == 0) store_part<DT, D>(p, it, w, part);
    return;
  }
  own_part<DT, D>(p, blockIdx.x - p.prefix_blocks, v);
}

// Many rows: a block takes NW * 32 rows of one cache head and a part of the
// prefix, each wave 32 rows; tiles of 64 slots go through LDS for all of them.
//
// Pipeline. While 32 slots' scores are turned into probabilities, the matrix
// units already make the next 32 slots' scores; the product with V follows. K
// therefore runs 32 slots ahead of V: a step works on V of slots k .. k + 63 and
// K of k + 32 .. k + 95. The next step's tiles are on their way meanwhile,
// straight from memory into the other half of LDS, with no registers in
// between: one barrier a step, where they have to have landed.
//
// LDS. A fetch writes 16 bytes a lane in lane order, so rows lie without
// padding and the lane picks which 16 bytes of its row it brings: piece c of
// row r lies at c ^ swizzle(r). The 64 banks serve 16 lanes of a 16-byte read
// at once (lanes 0-3, 12-15 and 20-27, or 4-11, 16-19 and 28-31) and 32 of an
// 8-byte one; the swizzles give each of them other banks.
//
// A wave fetches whole slots' rows, kGroup at a time; with pages of a multiple
// of kGroup slots they lie in one page. Lane g looks up the page of the wave's
// g-th group of the next step; the addresses are scalar arithmetic.
constexpr int kTile = 64;

template <int D>
constexpr int group_slots() {
  return D == 64 ? 8 : 4;
}
template <int D>
__device__ __forceinline__ int swizzle_k(int r) {
  return D == 128 ? r & 15 : D == 64 ? (r >> 1) & 7 : (r >> 2) & 3;
}
template <int D>
__device__ __forceinline__ int swizzle_v(int r) {
  return D == 128 ? 4 * (r & 3) : D == 64 ? 2 * (r & 2) : 0;
}

typedef __attribute__((address_space(3))) short lds_short;

// 16 bytes for each active lane from base + off into LDS at `at` + 16 * lane.
// The compiler does not see the transfer: the caller waits (wait_fetch) and
// passes a barrier before anyone reads.
__device__ __forceinline__ void fetch16(const void* base, uint32_t off, uint32_t at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(at), "v"(off), "s"(base)
               : "memory");
}
__device__ __forceinline__ void wait_fetch() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A wave's fetches of 32 slots ("half" a tile): kH groups of kGroup slots.
template <int D, int NW>
struct Fetch {
  static constexpr int kGroup = group_slots<D>();
  static constexpr int kH = 32 / (NW * kGroup);
  static_assert(kH >= 1 && NW * kGroup % 16 == 0, "every group of a wave swizzles alike");
  uint32_t koff, voff;  // the lane's byte offset in a group's rows
  bool on;              // the lane has a piece
  int wave;
  int page, in_page;    // of group g of the last two halves looked up, in lane g < 2 kH

  __device__ __forceinline__ void init(const PrefixDev& p) {
    const int lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane / (D / 8), c = lane % (D / 8);
    const int row = wave * kGroup + r;
    on = r < kGroup;
    koff = 2 * (uint32_t)(r * p.a.kv.kss + 8 * (c ^ swizzle_k<D>(row)));
    voff = 2 * (uint32_t)(r * p.a.kv.vss + 8 * (c ^ swizzle_v<D>(row)));
  }
  // Starts looking up the pages of the halves from slot0 and slot0 + 32. A
  // group past the end repeats the last one.
  __device__ __forceinline__ void look(const PrefixDev& p, const int* table, int slot0, int k1) {
    const int g = min(threadIdx.x & 63, 2 * kH - 1);
    const int at = slot0 + (g / kH) * 32 + (g % kH * NW + wave) * kGroup;
    const int slot = min(at, (k1 - 1) / kGroup * kGroup);
    const int col = div_by(p.a.kv.by_page, slot);
    page = table[col];
    in_page = slot - col * p.a.kv.page;
  }
  __device__ __forceinline__ void check(const PrefixDev& p) {
    if ((unsigned)page >= (unsigned)p.a.kv.pages) {
      flag(p, kKvBadPage);
      page = 0;
    }
  }
  // Fetches half `half` of those looked up, `at` being its place in LDS. ps and
  // ss are the strides of a page and a slot in 16 bytes.
  __device__ __forceinline__ void half_tile(const char* base, uint32_t ps, uint32_t ss, uint32_t off, int pages,
                                            int slots, int half, uint32_t at) const {
#pragma unroll
    for (int i = 0; i < kH; ++i) {
      const uint32_t pg = __builtin_amdgcn_readlane(pages, half * kH + i);
      const uint32_t sl = __builtin_amdgcn_readlane(slots, half * kH + i);
      const char* from = base + (((uint64_t)pg * ps + (uint64_t)(sl * ss)) << 4);
      if (on) fetch16(from, off, at + (i * NW + wave) * kGroup * 2 * D);
    }
  }
};

// The scores of 32 slots: K (rows of LDS at k) by the wave's queries.
template <int DT, int D>
__device__ __forceinline__ void scores(const Wave<DT, D>& w, const short* k, f16v (&s)[1]) {
  const int lane = threadIdx.x & 63, r = lane & 31;
  const int sw = swizzle_k<D>(r) ^ (lane >> 5);
  s[0] = f16v{};
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
    s[0] = mfma<DT>(*reinterpret_cast<const s8v*>(k + r * D + 8 * ((2 * i) ^ sw)), w.q[i], s[0]);
}

// The outputs' product with V (rows of LDS at v) of 32 slots.
template <int DT, int D>
__device__ __forceinline__ void times_v(Wave<DT, D>& w, const short* v, const s8v (&prob)[2]) {
  const int lane = threadIdx.x & 63, q = lane & 15;
  const int r = 4 * (lane >> 5) + (q >> 2);
  const int c = 2 * ((lane >> 4) & 1) + ((q & 3) >> 1), sw = swizzle_v<D>(r);  // the same for r + 8
#pragma unroll
  for (int kk = 0; kk < 2; ++kk)
#pragma unroll
    for (int d = 0; d < D / 32; ++d) {
      const short* at = v + (16 * kk + r) * D + 8 * ((4 * d + c) ^ sw) + 4 * (q & 1);
      const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)at);
      const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(at + 8 * D));
      w.o[d] = mfma<DT>(__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7), prob[kk], w.o[d]);
    }
}

template <int DT, int D, int NW>
__global__ __launch_bounds__(NW * 64, 2) void k_attend_wide(PrefixDev p) {
  using F = Fetch<D, NW>;
  constexpr int kRows = kTile * D;  // elements of a tile
  constexpr int kWide = 4 * kRows, kOwn = NW * v_tile_elems<D>();
  __shared__ __attribute__((aligned(1024))) short smem[kWide > kOwn ? kWide : kOwn];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if ((int)blockIdx.x >= p.prefix_blocks) {
    own_part<DT, D>(p, blockIdx.x - p.prefix_blocks, smem + wave * v_tile_elems<D>());
    return;
  }
  PrefixItem x;
  int part;
  // blocks are dealt to the 8 XCDs in turn: neighbours in the work's order,
  // which read the same part of the prefix, go to one XCD and its L2
  if (!prefix_item(p, xcd_remap(blockIdx.x, p.prefix_blocks), NW * 32, &x, &part)) return;
  const int k1 = x.k1;
  const KvView& kv = p.a.kv;
  Rows it = x.it;
  const char* kbase = kv.k + 2 * it.h * kv.khs;
  const char* vbase = kv.v + 2 * it.h * kv.vhs;
  it.r0 += 32 * wave;
  const bool live = it.r0 < it.rows;  // waves without rows only fetch
  Wave<DT, D> w;
  load_q<DT, D>(p, it, w);
  if (x.k0 < k1) {
    F f;
    f.init(p);
    const uint32_t lds = (uint32_t)(uintptr_t)(lds_short*)smem;
    // 32 slots' places: K 0 to 3 (two tiles), V 4 to 7
    auto at = [&](int i) { return lds + kRows * i; };
    auto fetch_k = [&](int half, int place) {
      f.half_tile(kbase, kv.kps >> 3, kv.kss >> 3, f.koff, f.page, f.in_page, half, at(place));
    };
    auto fetch_v = [&](int page, int in_page, int half, int place) {
      f.half_tile(vbase, kv.vps >> 3, kv.vss >> 3, f.voff, page, in_page, half, at(place));
    };
    f.look(p, x.pages, x.k0, k1);
    f.check(p);
    fetch_k(0, 2);
    fetch_k(1, 0);
    fetch_v(f.page, f.in_page, 0, 4);
    fetch_v(f.page, f.in_page, 1, 5);
    f.look(p, x.pages, x.k0 + 32, k1);
    f.check(p);
    fetch_k(1, 1);
    int vpage = f.page, vslot = f.in_page;  // the second half of these is the next one of V
    f.look(p, x.pages, x.k0 + 96, k1);
    wait_fetch();
    __syncthreads();
    f16v s[1], t[1];
    if (live) {
      scores<DT, D>(w, smem + kRows, s);  // its place becomes the second K tile's
      if (x.k0 + 32 > k1) mask_tile(s[0], x.k0, k1);
    }
    __syncthreads();
    // One step, on the tiles of parity b.
    auto step = [&](int k, int b) {
      const short* ks = smem + b * kRows;
      short* vs = smem + (2 + b) * kRows;
      if (k + kTile < k1) {
        f.check(p);  // slots k + 96 .. k + 159
        fetch_k(0, 2 - 2 * b);
        fetch_k(1, 3 - 2 * b);
        fetch_v(vpage, vslot, 1, 6 - 2 * b);
        fetch_v(f.page, f.in_page, 0, 7 - 2 * b);
        vpage = f.page;
        vslot = f.in_page;
        f.look(p, x.pages, k + 160, k1);
      } else if (k + kTile > k1) {
        // values behind the end are cleared: a probability of zero must not meet an infinity
        for (int i = threadIdx.x; i < (k + kTile - k1) * (D / 8); i += NW * 64)
          *reinterpret_cast<u4*>(vs + (k1 - k) * D + 8 * i) = u4{0, 0, 0, 0};
        __syncthreads();
      }
      if (live) {
        s8v prob[2];
        refer<DT, D, 1>(p, w, s);
        scores<DT, D>(w, ks, t);
        probabilities<DT, D, 1>(p, w, s, prob);
        times_v<DT, D>(w, vs, prob);
        if (k + 64 > k1) mask_tile(t[0], k + 32, k1);
        refer<DT, D, 1>(p, w, t);
        scores<DT, D>(w, ks + 32 * D, s);
        probabilities<DT, D, 1>(p, w, t, prob);
        times_v<DT, D>(w, vs + 32 * D, prob);
        if (k + 96 > k1) mask_tile(s[0], k + 64, k1);
      }
      wait_fetch();
      __syncthreads();
    };
    for (int k = x.k0; k < k1; k += 2 * kTile) {
      step(k, 0);
      if (k + kTile < k1) step(k + kTile, 1);
    }
  }
  if (live) store_part<DT, D>(p, it, w, part);
}

// Joins the parts of each (token, query head): 32 lanes, 4 columns each.
template <int DT, int D>
__global__ __launch_bounds__(256) void k_join(PrefixDev p) {
  const int l = threadIdx.x & 31;
  const long long rows = (long long)p.a.tokens * p.a.q_heads;
  const int parts = p.nps + p.nos;
  for (long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); row < rows; row += (long long)gridDim.x * 8) {
    float z0 = l < parts ? p.part_lse[l * rows + row] : kNegInf;
    float z1 = l + 32 < parts ? p.part_lse[(l + 32) * rows + row] : kNegInf;
    float top = fmaxf(z0, z1);
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 32));
    const float ref = top == kNegInf ? 0.f : top;
    z0 = __builtin_amdgcn_exp2f(z0 - ref);
    z1 = __builtin_amdgcn_exp2f(z1 - ref);
    float total = z0 + z1;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) total += __shfl_xor(total, d, 32);
    f4 acc = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < parts; ++i) {
      const float wgt = i < 32 ? __shfl(z0, i, 32) : __shfl(z1, i - 32, 32);
      if (wgt == 0.f) continue;  // an empty part holds nothing, not zeros
      if (l < D / 4) acc += *reinterpret_cast<const f4*>(p.part_o + (i * rows + row) * D + 4 * l) * wgt;
    }
    const bool some = !(total == 0.f);
    const float inv = some ? 1.f / total : 0.f;
    const long long t = row / p.a.q_heads;
    const int head = (int)(row - t * p.a.q_heads);
    if (l < D / 4) {
      u2 x;
      x.x = pack2<DT>(acc.x * inv, acc.y * inv);
      x.y = pack2<DT>(acc.z * inv, acc.w * inv);
      short* dst = reinterpret_cast<short*>(const_cast<void*>(p.a.out.p)) + t * p.a.out.ts + head * p.a.out.hs;
      *reinterpret_cast<u2*>(dst + 4 * l) = x;
    }
    if (l == 0 && p.a.lse) p.a.lse[row] = some ? (top + __log2f(total)) * 0.6931471805599453f : kNegInf;
  }
}

template <int DT, int D>
hipError_t launch(const PrefixDev& p, int blocks, bool wide, hipStream_t st) {
  if (wide) k_attend_wide<DT, D, 4><<<blocks, 256, 0, st>>>(p);
  else k_attend<DT, D><<<blocks, 256, 0, st>>>(p);
  if (hipError_t e = hipGetLastError()) return e;
  const long long rows = (long long)p.a.tokens * p.a.q_heads;
  k_join<DT, D><<<(unsigned)std::min<long long>((rows + 7) / 8, 1 << 20), 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_prefix_attention(const PrefixArgs& a, const PrefixPlan& plan, char* ws, hipStream_t st) {
  PrefixDev p{};
  p.a = a;
  // a scale of 0 would turn a masked -infinity into NaN; 1e-37 scales every
  // finite product of 16-bit operands to less than half a step of 1
  p.scale2 = std::max(std::fabs(a.scale) * 1.4426950408889634f, 1e-37f);
  p.q_sign = a.scale < 0.f ? 0x80008000u : 0u;
  p.m = a.q_heads / a.kv.heads;
  p.by_m = fast_div((uint32_t)p.m);
  p.nps = plan.nps;
  p.nos = plan.nos;
  p.prefix_tiles = (int)plan.prefix_tiles;
  p.prefix_blocks = (int)plan.prefix_blocks;
  p.own_tq = plan.own_tq;
  p.own_tiles = (int)plan.own_tiles;
  p.part_o = reinterpret_cast<float*>(ws + plan.o_off);
  p.part_lse = reinterpret_cast<float*>(ws + plan.lse_off);
  const int blocks = (int)(plan.prefix_blocks + plan.own_blocks);
  const bool bf = a.kv.dtype == EMB_BF16;
  switch (a.kv.dim) {
    case 64: return bf ? launch<EMB_BF16, 64>(p, blocks, plan.wide, st) : launch<EMB_F16, 64>(p, blocks, plan.wide, st);
    case 96: return bf ? launch<EMB_BF16, 96>(p, blocks, plan.wide, st) : launch<EMB_F16, 96>(p, blocks, plan.wide, st);
    default: return bf ? launch<EMB_BF16, 128>(p, blocks, plan.wide, st) : launch<EMB_F16, 128>(p, blocks, plan.wide, st);
  }
}

}  // namespace emb
