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
//
// Measured: 1024 queries over 32768 slots (32 x 8 heads of 128) 555 us, 990
// TFLOP/s, where a large library product reaches 1391; the matrix units are
// busy half of the cycles, at 1.85 GHz. 24 groups' 2400 queries over prefixes of
// 512 to 2048 and 20 own slots 101 us (2.5 TB/s), 509 queries over 8191 slots
// (16 heads of 64) 44 us, 8 over 4096 slots 21 us: the last two are chains of
// dependent reads (offsets, lengths, pages, keys) and two launches. Own
// sequences alone: 64 queries over 2000 slots each 111 us (4.7 TB/s), a prompt
// of 2000 queries 170 us (195 TFLOP/s: each wave reads its sequence's slots for
// itself).
#include <algorithm>
#include <cmath>

#include "seq_device.h"

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
  bool zero;     // the scale is 0
  uint32_t q_sign;  // sign bits of two elements where the scale is negative
  int m;         // query heads of a cache head
  FastDiv by_m;
  int nps, nos;
  int prefix_blocks, prefix_tiles;  // tiles: upper bound, blocks = tiles * heads * nps
  int own_tiles;                    // tiles of 32 rows
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

// 0 for each finite element, NaN for the others.
template <int DT>
__device__ __forceinline__ u4 times_zero(u4 x) {
  constexpr uint32_t top = DT == EMB_BF16 ? 0x7f80u : 0x7c00u;
  auto one = [](uint32_t w) {
    return ((w & top) == top ? 0x7fffu : 0u) | ((w >> 16 & top) == top ? 0x7fff0000u : 0u);
  };
  return u4{one(x.x), one(x.y), one(x.z), one(x.w)};
}

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
  if (p.zero) {  // once, behind all of the loads
#pragma unroll
    for (int s = 0; s < D / 16; ++s) w.q[s] = __builtin_bit_cast(s8v, times_zero<DT>(__builtin_bit_cast(u4, w.q[s])));
  }
#pragma unroll
  for (int d = 0; d < D / 32; ++d) w.o[d] = f16v{};
  w.mx = kNegInf;
  w.sum = 0.f;
}

// Slot `slot` of a page table row, without a check of the page.
__device__ __forceinline__ int page_of(const PrefixDev& p, const int* pages, int slot, int* in_page) {
  const int col = div_by(p.a.kv.by_page, slot);
  *in_page = slot - col * p.a.kv.page;
  return pages[col];
}
// A slot without a page reads page 0 and raises the flag (its values are then
// meaningless, but in range).
__device__ __forceinline__ int checked(const PrefixDev& p, int page) {
  if ((unsigned)page < (unsigned)p.a.kv.pages) return page;
  flag(p, kKvBadPage);
  return 0;
}

// Elements between rows of a wave's own V tile: 4 rows, 64 bytes of each, are
// read at once and have to lie in different banks of the 64.
template <int D>
constexpr int v_pad() {
  return D == 96 ? 0 : 32;
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
// keeps the probabilities below 2^15. Each row goes by its own scores alone.
template <int DT, int D>
__device__ __forceinline__ void refer(const PrefixDev& p, Wave<DT, D>& w, float lane_top) {
  const float top = both_halves_max(lane_top) * p.scale2;
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

// The keys of slot lane % 32 of a tile, and the values of the lane's pieces,
// from (page, slot in it) of the lane's slot.
template <int D>
constexpr int kPieces = 32 * D / 8 / 64;  // 16-byte pieces of a V tile for each lane

template <int D>
__device__ __forceinline__ void load_k(const KvView& kv, int page, int in_page, int h, s8v (&kf)[D / 16]) {
  const short* kp = reinterpret_cast<const short*>(kv.k) + page * kv.kps + in_page * kv.kss + h * kv.khs;
#pragma unroll
  for (int s = 0; s < D / 16; ++s)
    kf[s] = *reinterpret_cast<const s8v*>(kp + 16 * s + 8 * ((threadIdx.x & 63) >> 5));
}
template <int D>
__device__ __forceinline__ void load_v(const KvView& kv, int page, int in_page, int h, s8v (&vr)[kPieces<D>]) {
#pragma unroll
  for (int i = 0; i < kPieces<D>; ++i) {
    const int piece = i * 64 + (threadIdx.x & 63), row = piece / (D / 8);
    const int pg = __shfl(page, row, 64), sl = __shfl(in_page, row, 64);
    vr[i] = *reinterpret_cast<const s8v*>(reinterpret_cast<const short*>(kv.v) + pg * kv.vps + sl * kv.vss +
                                          h * kv.vhs + 8 * (piece % (D / 8)));
  }
}
// Into the wave's LDS tile; rows outside [lo, hi) as zeros.
template <int D>
__device__ __forceinline__ void put_v(short* v, const s8v (&vr)[kPieces<D>], int lo, int hi) {
#pragma unroll
  for (int i = 0; i < kPieces<D>; ++i) {
    const int piece = i * 64 + (threadIdx.x & 63), row = piece / (D / 8);
    *reinterpret_cast<s8v*>(v + row * (D + v_pad<D>()) + 8 * (piece % (D / 8))) =
        row >= lo && row < hi ? vr[i] : s8v{};
  }
}

// One wave over the prefix slots k0, k0 + step, .. below k1 in tiles of 32, the
// keys straight into registers (each is used once) and the values through the
// wave's own LDS tile. next_page, next_in: the first tile's, from first_page.
__device__ __forceinline__ int first_page(const PrefixDev& p, const int* pages, int k, int k1, int* in_page) {
  // slots past the end read the last one again; their scores are masked
  return page_of(p, pages, min(k + (int)(threadIdx.x & 31), k1 - 1), in_page);
}
template <int DT, int D>
__device__ void wave_slots(const PrefixDev& p, Wave<DT, D>& w, const int* pages, int h, int k0, int k1, int step,
                           short* v, int next_page, int next_in) {
#pragma unroll 1
  for (int k = k0; k < k1; k += step) {
    const int page = checked(p, next_page), in_page = next_in;
    s8v kf[D / 16], vr[kPieces<D>];
    load_k<D>(p.a.kv, page, in_page, h, kf);
    load_v<D>(p.a.kv, page, in_page, h, vr);
    if (k + step < k1) next_page = first_page(p, pages, k + step, k1, &next_in);
    f16v s[1] = {};
#pragma unroll
    for (int i = 0; i < D / 16; ++i) s[0] = mfma<DT>(kf[i], w.q[i], s[0]);
    // values behind the end are cleared: a probability of zero must not meet an infinity
    put_v<D>(v, vr, 0, k1 - k);
    __builtin_amdgcn_sched_barrier(0);
    s8v prob[2];
    if (k + 32 > k1) mask_tile(s[0], k, k1);
    refer<DT, D>(p, w, top_of(s));
    probabilities<DT, D, 1>(p, w, s, prob);
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) w.o[d] = mfma<DT>(read_vt<D>(v, 16 * kk, 32 * d), prob[kk], w.o[d]);
  }
}

// ---- values in LDS as fetches leave them: 16-byte piece c of row r at c ^ swizzle(r)

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
// `at` is an operand in m0, so the compiler knows what the register holds. It
// does not see the transfer: the caller waits (wait_fetch) and passes a barrier
// before anyone reads. It does not see the instruction's hazards either: a base
// that a vector instruction wrote would have to be five wait states old, so a
// scalar one copies it, and that copy is the wait state which m0 needs.
__device__ __forceinline__ void fetch16(uint64_t base, uint32_t off, uint32_t at) {
  uint64_t from;
  asm volatile("s_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0"
               : "=&s"(from)
               : "{m0}"(at), "v"(off), "s"(base)
               : "memory");
}
__device__ __forceinline__ void wait_fetch() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
// Before a wave fetches into LDS that it has read itself: its reads are over.
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// The same with an address for each lane.
__device__ __forceinline__ void fetch16(uint64_t from, uint32_t at) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
               :
               : "{m0}"(at), "v"(from)
               : "memory");
}

// V^T operand of 16 slots from slot 16 kk and 32 columns from 32 d (rows of LDS at v).
template <int D>
__device__ __forceinline__ s8v operand_v(const short* v, int kk, int d) {
  const int lane = threadIdx.x & 63, q = lane & 15;
  const int r = 4 * (lane >> 5) + (q >> 2);
  const int c = 2 * ((lane >> 4) & 1) + ((q & 3) >> 1), sw = swizzle_v<D>(r);  // the same for r + 8
  const short* at = v + (16 * kk + r) * D + 8 * ((4 * d + c) ^ sw) + 4 * (q & 1);
  const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)at);
  const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(at + 8 * D));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// The outputs' product with V of 16 slots.
template <int DT, int D>
__device__ __forceinline__ void times_v(Wave<DT, D>& w, const short* v, int kk, const s8v& prob) {
#pragma unroll
  for (int d = 0; d < D / 32; ++d) w.o[d] = mfma<DT>(operand_v<D>(v, kk, d), prob, w.o[d]);
}

// ---- own sequences ---------------------------------------------------------
// The 32 rows of a tile belong to one sequence or to several. Each sequence is
// taken in tiles of 32 slots by all rows, those of other sequences masked: such
// tiles wait for their reads, and products of masked rows cost nothing on top.
// The sequences' tiles form one list, so that the next tile's page is looked up while this one
// is worked on. With several waves to share it, tile t of sequence b goes to
// wave (b + t) % step: where a sequence is cut does not depend on its
// neighbours, and neither does a bit of its result.

// Row lane % 32 of the tile.
struct OwnRow {
  int b;      // its sequence
  int seen;   // slots the row sees
  int first;  // the sequence's first tile of this wave
  int base;   // tiles of this wave before the sequence's
  int end;    // behind its tiles for the last row of a sequence, base for its others
};

// The last i in [lo, hi) with f(i) <= x for each lane, f non-decreasing, f(lo) <= x.
template <class F>
__device__ __forceinline__ int lane_find(int lo, int hi, int x, F f) {
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (f(mid) <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// s0, s1: the sequences among which the tile's rows are.
__device__ __forceinline__ OwnRow own_row(const PrefixDev& p, const Rows& it, int s0, int s1, int i0, int step) {
  const int lane = threadIdx.x & 63;
  const int row = it.r0 + (lane & 31);
  const int tok = it.t0 + div_by(p.by_m, min(row, it.rows - 1));
  OwnRow r;
  int first = tok, n = 1;
  r.b = tok;
  if (p.a.offsets) {
    const int tok0 = __builtin_amdgcn_readlane(tok, 0), tok1 = __builtin_amdgcn_readlane(tok, 31);
    // 64 sequences' first tokens in the lanes, from the tile's first one
    int b0 = s0;
    if (s1 - s0 >= 64) b0 += wave_find(s1 - s0, tok0, [&](int i) { return first_token(p, s0 + i); });
    const int off = first_token(p, min(b0 + lane, p.a.seqs));
    if (b0 + 63 >= s1 || __builtin_amdgcn_readlane(off, 63) > tok1) {
      int at = 0;
#pragma unroll
      for (int d = 32; d >= 1; d >>= 1) {
        const int x = __shfl(off, at + d, 64);
        if (at + d < 64 && b0 + at + d < s1 && x <= tok) at += d;
      }
      r.b = b0 + at;
      first = __shfl(off, at, 64);
      n = __shfl(off, min(at + 1, 63), 64) - first;
    } else {  // many empty sequences among them
      r.b = lane_find(b0, s1, tok, [&](int i) { return first_token(p, i); });
      first = first_token(p, r.b);
      n = first_token(p, min(r.b + 1, p.a.seqs)) - first;
    }
    r.b = min(r.b, p.a.seqs - 1);
  }
  int len = p.a.lens[r.b];
  const long long cap = (long long)p.a.width * p.a.kv.page;
  if (len < 0 || len > cap) {
    if (row < it.rows) flag(p, kKvBadPage);
    len = len < 0 ? 0 : (int)cap;
  }
  const bool in = row < it.rows && tok >= first && tok < first + n;
  r.seen = in ? max(len - n + tok - first + 1, 0) : 0;
  r.first = i0 - (r.b - s0) % step;
  if (r.first < 0) r.first += step;
  // the last row of a sequence, which sees the most, carries its tiles; running sums over the rows
  const int next = __shfl_down(r.b, 1, 64);
  const bool last = (lane & 31) == 31 || next != r.b || row + 1 >= it.rows;
  const int tiles = (r.seen + 31) / 32;
  const int own = last && tiles > r.first ? (tiles - r.first + step - 1) / step : 0;
  r.end = own;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int x = __shfl_up(r.end, d, 32);
    if ((lane & 31) >= d) r.end += x;
  }
  r.base = r.end - own;
  return r;
}

// Whether any of the wave's 32 rows of D values at v holds an infinity or NaN.
template <int DT, int D>
__device__ __forceinline__ bool any_special(const short* v) {
  typedef unsigned short us8 __attribute__((ext_vector_type(8)));
  us8 top = {};
#pragma unroll
  for (int i = 0; i < kPieces<D>; ++i)
    top = __builtin_elementwise_max(
        top, *reinterpret_cast<const us8*>(v + 8 * (i * 64 + (threadIdx.x & 63))) & (unsigned short)0x7fff);
  typedef unsigned short us4 __attribute__((ext_vector_type(4)));
  typedef unsigned short us2 __attribute__((ext_vector_type(2)));
  const us4 t4 = __builtin_elementwise_max(top.lo, top.hi);
  const us2 t2 = __builtin_elementwise_max(t4.lo, t4.hi);
  return __ballot(max(t2.x, t2.y) >= (DT == EMB_BF16 ? 0x7f80 : 0x7c00));
}

// Tile i of the wave's list.
struct OwnTile {
  int b, slot0, lim;  // uniform: the sequence, the first slot, the rows' largest limit
  int page, in_page;  // of slot lane % 32; slots from lim on repeat the last one below
};
__device__ __forceinline__ int own_total(const OwnRow& r) { return __builtin_amdgcn_readlane(r.end, 31); }
// All but the page; its column of the sequence's page table row.
__device__ __forceinline__ int own_place(const PrefixDev& p, const OwnRow& r, int i, int step, OwnTile* t) {
  const int at = __ffsll((unsigned long long)(uint32_t)__ballot(r.end > i)) - 1;
  t->b = __builtin_amdgcn_readlane(r.b, at);
  t->slot0 = 32 * (__builtin_amdgcn_readlane(r.first, at) + (i - __builtin_amdgcn_readlane(r.base, at)) * step);
  t->lim = __builtin_amdgcn_readlane(r.seen, at);
  const int slot = min(t->slot0 + (int)(threadIdx.x & 31), t->lim - 1);
  const int col = div_by(p.a.kv.by_page, slot);
  t->in_page = slot - col * p.a.kv.page;
  return col;
}
__device__ __forceinline__ OwnTile own_look(const PrefixDev& p, const OwnRow& r, int i, int step) {
  OwnTile t;
  const int col = own_place(p, r, i, step, &t);
  t.page = (p.a.table + (long long)t.b * p.a.width)[col];
  return t;
}

// The wave's tiles into w, the first one given. A zero probability must not meet
// an infinity or NaN that its row does not see (0 * infinity), so tiles with such
// values are left out (the return value tells) and taken by a second call with
// WINDOWS: one product for each limit among the sequence's rows with the values
// beyond it cleared, of which each row keeps its own. The products add to the outputs
// as the first call's do, and a tile with values that a row does not see is that row's
// last one: every bit is what it is without them.
template <int DT, int D, bool WINDOWS>
__device__ __forceinline__ bool own_tiles(const PrefixDev& p, Wave<DT, D>& w, const OwnRow& r, OwnTile next, int h,
                                          int step, short* v) {
  const int lane = threadIdx.x & 63;
  const KvView& kv = p.a.kv;
  const int total = own_total(r);
  const uint32_t lds = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_short*)v);
  // a tile's keys into registers, its values into half `buf` of the wave's LDS
  auto fetch = [&](OwnTile& t, s8v (&kf)[D / 16], int buf) {
    t.page = checked(p, t.page);
    load_k<D>(kv, t.page, t.in_page, h, kf);
    const uint64_t from = (uint64_t)(kv.v + 2 * (t.page * kv.vps + t.in_page * kv.vss + h * kv.vhs));
    const int lo = (int)from, hi = (int)(from >> 32);
#pragma unroll
    for (int i = 0; i < kPieces<D>; ++i) {
      const int piece = i * 64 + lane, row = piece / (D / 8), c = piece % (D / 8) ^ swizzle_v<D>(row);
      const uint64_t at = (uint64_t)(uint32_t)__shfl(hi, row, 64) << 32 | (uint32_t)__shfl(lo, row, 64);
      fetch16(at + 16 * c, lds + buf * 64 * D + i * 1024);
    }
  };
  bool left = false;
  OwnTile t = next;
  s8v kf[D / 16], kn[D / 16];
  wait_reads();
  fetch(t, kf, 0);
  if (total > 1) next = own_look(p, r, 1, step);
#pragma unroll 1
  for (int i = 0; i < total; ++i) {
    short* vt = v + (i & 1) * 32 * D;
    const OwnTile now = t;
    f16v s[1] = {};
#pragma unroll
    for (int c = 0; c < D / 16; ++c) s[0] = mfma<DT>(kf[c], w.q[c], s[0]);
    wait_fetch();
    if (i + 1 < total) {
      t = next;
      wait_reads();
      fetch(t, kn, (i + 1) & 1);
      if (i + 2 < total) next = own_look(p, r, i + 2, step);
    }
#pragma unroll
    for (int c = 0; c < D / 16; ++c) kf[c] = kn[c];
    const bool special = any_special<DT, D>(vt);
    if (special != WINDOWS) {
      left = true;
      continue;
    }
    const bool mine = r.b == now.b;
    mask_tile(s[0], now.slot0, mine ? r.seen : 0);
    s8v prob[2];
    refer<DT, D>(p, w, top_of(s));
    probabilities<DT, D, 1>(p, w, s, prob);
    if (!WINDOWS) {
      times_v<DT, D>(w, vt, 0, prob[0]);
      times_v<DT, D>(w, vt, 1, prob[1]);
      continue;
    }
    int done = 1 << 30;  // limits from this one on are through
    for (int a = 31; a >= 0; --a) {
      const int lim = __builtin_amdgcn_readlane(r.seen, a);
      if (__builtin_amdgcn_readlane(r.b, a) != now.b || lim >= done || lim <= now.slot0) continue;
      done = lim;
#pragma unroll
      for (int c = 0; c < kPieces<D>; ++c) {
        const int piece = c * 64 + lane;
        if (now.slot0 + piece / (D / 8) >= lim) *reinterpret_cast<s8v*>(vt + 8 * piece) = s8v{};
      }
      const bool takes = mine && r.seen == lim;
#pragma unroll
      for (int d = 0; d < D / 32; ++d) {
        f16v o = w.o[d];
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) o = mfma<DT>(operand_v<D>(vt, kk, d), prob[kk], o);
#pragma unroll
        for (int c = 0; c < 16; ++c) w.o[d][c] = takes ? o[c] : w.o[d][c];
      }
    }
  }
  return left;
}

// What the wave has to do of the rows' own slots, into w. `page`: of the first
// tile's slots (own_look's), where there is one.
template <int DT, int D>
__device__ __forceinline__ void own_slots(const PrefixDev& p, Wave<DT, D>& w, const OwnRow& r, int page, int h, int step,
                                          short* v) {
  if (own_total(r) == 0) return;
  OwnTile t;
  own_place(p, r, 0, step, &t);
  t.page = page;
  if (own_tiles<DT, D, false>(p, w, r, t, h, step, v)) own_tiles<DT, D, true>(p, w, r, own_look(p, r, 0, step), h, step, v);
}

// Stores the wave's rows: as partial output `part`, or, where there is only one
// part, as the call's result.
template <int DT, int D>
__device__ __forceinline__ void store_rows(const PrefixDev& p, const Rows& it, Wave<DT, D>& w, int part) {
  const int lane = threadIdx.x & 63;
  const int row = it.r0 + (lane & 31);
  const float total = both_halves_sum(w.sum);
  const bool some = !(total == 0.f);  // a NaN counts
  const float z = some ? w.mx - kShift + __log2f(total) : kNegInf;
  const float inv = some ? 1.f / total : 0.f;
  const int j = div_by(p.by_m, min(row, it.rows - 1));
  const int head = it.h * p.m + min(row, it.rows - 1) - j * p.m;
  if (p.nps + p.nos == 1) {
    const long long at = (long long)(it.t0 + j) * p.a.q_heads + head;
    if (row < it.rows && lane < 32 && p.a.lse) p.a.lse[at] = some ? z * 0.6931471805599453f : kNegInf;
    short* dst = reinterpret_cast<short*>(const_cast<void*>(p.a.out.p)) + (long long)(it.t0 + j) * p.a.out.ts +
                 head * p.a.out.hs + 8 * (lane >> 5);
    // lanes l and l + 32 hold 4 columns each of every 8; they trade halves so
    // that one stores columns 16 i .. + 7 and the other the next 8
    typedef unsigned u2v __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const f16v& o = w.o[d];
        const u2v lo = __builtin_amdgcn_permlane32_swap(pack2<DT>(o[8 * i] * inv, o[8 * i + 1] * inv),
                                                        pack2<DT>(o[8 * i + 4] * inv, o[8 * i + 5] * inv), false, false);
        const u2v hi = __builtin_amdgcn_permlane32_swap(pack2<DT>(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                                        pack2<DT>(o[8 * i + 6] * inv, o[8 * i + 7] * inv), false, false);
        if (row < it.rows) *reinterpret_cast<u4*>(dst + 32 * d + 16 * i) = some ? u4{lo.x, hi.x, lo.y, hi.y} : u4{0, 0, 0, 0};
      }
    return;
  }
  if (row >= it.rows) return;
  const long long at = ((long long)part * p.a.tokens + it.t0 + j) * p.a.q_heads + head;
  if (lane < 32) p.part_lse[at] = z;
  if (!some) return;
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
  int s0, s1;  // the group's sequences
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
  const long long cap = (long long)p.a.pwidth * p.a.kv.page;
  auto limit = [&](int n) { return n < 0 ? 0 : (int)min((long long)n, cap); };  // check_sequences reports others
  int g, t0, t1, len;
  if (p.a.groups <= 64) {
    // A group for each lane; tiles in the order of falling prefix lengths, so
    // that the longest are not the last to start.
    const int lane = threadIdx.x & 63, i = min(lane, p.a.groups - 1);
    const int l = limit(p.a.prefix_lens[i]);
    const int c0 = min(max(p.a.group_offsets[i], 0), p.a.seqs), c1 = min(max(p.a.group_offsets[i + 1], 0), p.a.seqs);
    const int a0 = first_token(p, c0), a1 = first_token(p, c1);
    const int n = lane < p.a.groups && a1 > a0 ? ((a1 - a0) * p.m + rows - 1) / rows : 0;
    int at = 0;  // tiles before this group's
    const int order = (int)((uint32_t)l >> 5 << 6) + 63 - lane;
    for (int j = 0; j < p.a.groups; ++j) {
      const int nj = __builtin_amdgcn_readlane(n, j);
      at += __builtin_amdgcn_readlane(order, j) > order ? nj : 0;
    }
    const uint64_t mine = __ballot(tile >= at && tile < at + n);
    if (!mine) return false;
    g = __ffsll((unsigned long long)mine) - 1;
    t0 = __builtin_amdgcn_readlane(a0, g);
    t1 = __builtin_amdgcn_readlane(a1, g);
    len = __builtin_amdgcn_readlane(l, g);
    w->s0 = __builtin_amdgcn_readlane(c0, g);
    w->s1 = __builtin_amdgcn_readlane(c1, g);
    w->it = Rows{t0, (tile - __builtin_amdgcn_readlane(at, g)) * rows, (t1 - t0) * p.m, h};
  } else {
    // tile i of the group whose tiles start at g + (its first row) / rows: a
    // bound that counts more tiles than there are
    g = wave_find(p.a.groups, tile, [&](int i) { return i + group_token(p, i) * p.m / rows; });
    t0 = group_token(p, g);
    t1 = group_token(p, g + 1);
    w->it = Rows{t0, (tile - (g + t0 * p.m / rows)) * rows, (t1 - t0) * p.m, h};
    if (w->it.r0 < 0 || w->it.r0 >= w->it.rows) return false;
    len = limit(p.a.prefix_lens[g]);
    w->s0 = min(max(p.a.group_offsets[g], 0), p.a.seqs);
    w->s1 = min(max(p.a.group_offsets[g + 1], 0), p.a.seqs);
  }
  const int chunk = max(128, ((len + p.nps - 1) / p.nps + 127) & ~127);
  w->k0 = (int)min((long long)*part * chunk, (long long)len);
  w->k1 = min(w->k0 + chunk, len);
  w->pages = p.a.prefix_table + (long long)g * p.a.pwidth;
  return true;
}

// Own sequences on their own: each wave of block `block` for itself takes a tile
// of 32 rows, a cache head and a part of the rows' own slots; part fastest,
// then the tile, then the cache head. False where there is none.
__device__ __forceinline__ bool own_item(const PrefixDev& p, int block, Rows* it, int* part) {
  int id = block * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  *part = id % p.nos;
  id /= p.nos;
  const int tile = id % p.own_tiles;
  const int h = id / p.own_tiles;
  *it = Rows{0, tile * 32, p.a.tokens * p.m, h};
  return h < p.a.kv.heads;
}

// Reports offsets that break their contract and prefixes that their tables do
// not hold, spread over the grid.
__device__ __forceinline__ void check_sequences(const PrefixDev& p) {
  if (p.a.offsets) report_offsets(p.a.offsets, p.a.seqs, p.a.tokens, p.a.kv.error);
  if (!p.a.kv.error) return;
  const long long cap = (long long)p.a.pwidth * p.a.kv.page;
  for (long long g = (long long)blockIdx.x * 256 + threadIdx.x; g < p.a.groups; g += (long long)gridDim.x * 256) {
    const int a = p.a.group_offsets[g], b = p.a.group_offsets[g + 1], len = p.a.prefix_lens[g];
    const int bits = (breaks_offsets(a, b, g, p.a.groups, p.a.seqs) ? kKvBadOffsets : 0) |
                     (len < 0 || len > cap ? kKvBadPage : 0);
    if (bits) flag(p, bits);
  }
}

// Few rows: a block takes one tile of 32 rows, a cache head and a part of the
// prefix; its four waves take every fourth tile of slots and are joined in LDS.
template <int DT, int D>
__global__ __launch_bounds__(256, 2) void k_attend(PrefixDev p) {
  constexpr int OS = D + 4;  // row stride of the joined outputs (floats): rows start 4 banks apart
  constexpr size_t kV = 4 * 64 * D * sizeof(short), kO = (2 * 32 * OS + 4 * 64) * sizeof(float);
  __shared__ __attribute__((aligned(16))) char smem[kV > kO ? kV : kO];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  short* v = reinterpret_cast<short*>(smem) + wave * 64 * D;
  Wave<DT, D> w;
  check_sequences(p);
  const bool prefix = (int)blockIdx.x < p.prefix_blocks;
  PrefixItem x;
  int part;
  if (prefix) {
    if (!prefix_item(p, blockIdx.x, 32, &x, &part)) return;
  } else {
    if (!own_item(p, blockIdx.x - p.prefix_blocks, &x.it, &part)) return;
    x.s0 = 0;
    x.s1 = p.a.seqs;
  }
  const Rows it = x.it;
  const int k0 = prefix ? x.k0 + 32 * wave : 0, k1 = prefix ? x.k1 : 0;
  // what the first prefix tile and the own slots need is looked up at once
  int first = 0, first_in = 0;
  if (k0 < k1) first = first_page(p, x.pages, k0, k1, &first_in);
  load_q<DT, D>(p, it, w);
  const bool own = !prefix || p.nos == 0;
  const int step = prefix ? p.nps * 4 : p.nos;
  OwnRow r;
  int page = 0;
  if (own) {
    r = own_row(p, it, x.s0, x.s1, prefix ? part * 4 + wave : part, step);
    if (own_total(r) > 0) page = own_look(p, r, 0, step).page;
  }
  if (prefix) wave_slots<DT, D>(p, w, x.pages, it.h, k0, k1, 128, v, first, first_in);
  if (own) own_slots<DT, D>(p, w, r, page, it.h, step, v);
  if (prefix) {
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
    if (wave > 0) return;
  }
  store_rows<DT, D>(p, it, w, prefix ? part : p.nps + part);
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
// of kGroup slots they lie in one page. The lanes look up the pages of the
// wave's next 64 groups at once and hold their addresses for the fetches.
constexpr int kTile = 64;

template <int D>
constexpr int group_slots() {
  return D == 64 ? 8 : 4;
}


// A wave's fetches of 32 slots ("half" a tile): kH groups of kGroup slots. Lane l
// holds the addresses of group l % kH of half l / kH - 1 of a window of 64 / kH
// halves.
template <int D, int NW>
struct Fetch {
  static constexpr int kGroup = group_slots<D>();
  static constexpr int kH = 32 / (NW * kGroup);
  static constexpr int kPairs = 32 / kH;  // of halves, in a window
  static_assert(NW == 4 && kH >= 1 && NW * kGroup % 16 == 0, "every group of a wave swizzles alike");
  struct Half {
    uint64_t k[kH], v[kH];  // uniform: where its groups' rows are
  };
  uint32_t koff, voff;  // the lane's byte offset in a group's rows
  bool on;              // the lane has a piece
  int wave;
  uint64_t k, v;        // of the window in use
  int page, in_page;    // of the next one
  int pair, window;     // the next pair of the window in use; the last window looked up

  __device__ __forceinline__ void init(const PrefixDev& p) {
    const int lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane / (D / 8), c = lane % (D / 8);
    const int row = wave * kGroup + r;
    on = r < kGroup;
    koff = 2 * (uint32_t)(r * p.a.kv.kss + 8 * (c ^ swizzle_k<D>(row)));
    voff = 2 * (uint32_t)(r * p.a.kv.vss + 8 * (c ^ swizzle_v<D>(row)));
    k = v = 0;
    page = in_page = pair = window = 0;
  }
  // Starts looking up the pages of window `window` of the slots [k0, k1). A
  // group past the end repeats the last one.
  __device__ __forceinline__ void look(const PrefixDev& p, const int* table, int k0, int k1) {
    const int l = threadIdx.x & 63;
    const long long at = k0 + (2 * kPairs * (long long)window + l / kH - 1) * 32 + (l % kH * NW + wave) * kGroup;
    const int slot = (int)min(max(at, (long long)k0), (long long)((k1 - 1) / kGroup * kGroup));
    page = page_of(p, table, slot, &in_page);
  }
  __device__ __forceinline__ void turn_to_next(const PrefixDev& p, int h) {
    const KvView& kv = p.a.kv;
    page = checked(p, page);
    k = (uint64_t)(kv.k + 2 * (page * kv.kps + in_page * kv.kss + h * kv.khs));
    v = (uint64_t)(kv.v + 2 * (page * kv.vps + in_page * kv.vss + h * kv.vhs));
  }
  static __device__ __forceinline__ uint64_t lane_of(uint64_t x, int l) {
    const uint32_t lo = __builtin_amdgcn_readlane((int)x, l), hi = __builtin_amdgcn_readlane((int)(x >> 32), l);
    return (uint64_t)hi << 32 | lo;
  }
  // The next two halves.
  __device__ __forceinline__ void take(const PrefixDev& p, const int* table, int h, int k0, int k1, Half* a, Half* b) {
    if (pair == kPairs) {
      pair = 0;
      turn_to_next(p, h);
    }
    if (pair == kPairs / 2) {
      ++window;
      look(p, table, k0, k1);
    }
#pragma unroll
    for (int i = 0; i < kH; ++i) {
      a->k[i] = lane_of(k, 2 * pair * kH + i);
      a->v[i] = lane_of(v, 2 * pair * kH + i);
      b->k[i] = lane_of(k, (2 * pair + 1) * kH + i);
      b->v[i] = lane_of(v, (2 * pair + 1) * kH + i);
    }
    ++pair;
  }
  // Fetches a half's rows into LDS at `at`.
  __device__ __forceinline__ void rows(const uint64_t (&from)[kH], uint32_t off, uint32_t at) const {
#pragma unroll
    for (int i = 0; i < kH; ++i)
      if (on) fetch16(from[i], off, at + (i * NW + wave) * kGroup * 2 * D);
  }
};

// The wave's operands of 32 slots' keys (rows of LDS at k).
template <int D>
__device__ __forceinline__ void read_k(const short* k, s8v (&kf)[D / 16]) {
  const int lane = threadIdx.x & 63, r = lane & 31;
  const int sw = swizzle_k<D>(r) ^ (lane >> 5);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) kf[i] = *reinterpret_cast<const s8v*>(k + r * D + 8 * ((2 * i) ^ sw));
}

// 32 slots: their scores `s` (maximum `top`) become probabilities and meet V,
// while the matrix units make the next 32 slots' scores `t` of the keys kf. NEXT:
// kf then takes the keys at k. The wave goes first on its SIMD from the first
// product to the last, so that the two waves there take turns with products and
// scalar work instead of mixing them (1024 candidates over 32768 slots 600 ->
// 572 us; sequences given with sched_group_barrier measured the same as the
// compiler's own).
template <int DT, int D, bool NEXT>
__device__ __forceinline__ void half_step(const PrefixDev& p, Wave<DT, D>& w, f16v (&s)[1], f16v (&t)[1], float& top,
                                          s8v (&kf)[D / 16], const short* v, const short* k) {
  refer<DT, D>(p, w, top);
  __builtin_amdgcn_s_setprio(1);
  t[0] = f16v{};
#pragma unroll
  for (int i = 0; i < D / 16; ++i) t[0] = mfma<DT>(kf[i], w.q[i], t[0]);
  s8v prob[2];
  probabilities<DT, D, 1>(p, w, s, prob);
  times_v<DT, D>(w, v, 0, prob[0]);
  if (NEXT) read_k<D>(k, kf);
  times_v<DT, D>(w, v, 1, prob[1]);
  __builtin_amdgcn_s_setprio(0);
  top = top_of(t);
}

template <int DT, int D, int NW>
__global__ __launch_bounds__(NW * 64, 2) void k_attend_wide(PrefixDev p) {
  using F = Fetch<D, NW>;
  constexpr int kRows = kTile * D;  // elements of a tile
  __shared__ __attribute__((aligned(1024))) short smem[4 * kRows];  // own tiles: 64 rows for each wave
  __shared__ OwnRow s_own[NW][32];
  __shared__ int s_page[NW][32];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  check_sequences(p);
  const bool prefix = (int)blockIdx.x < p.prefix_blocks;
  PrefixItem x;
  int part;
  if (prefix) {
    // blocks are dealt to the 8 XCDs in turn: neighbours in the work's order,
    // which read the same part of the prefix, go to one XCD and its L2
    if (!prefix_item(p, xcd_remap(blockIdx.x, p.prefix_blocks), NW * 32, &x, &part)) return;
  } else {
    if (!own_item(p, blockIdx.x - p.prefix_blocks, &x.it, &part)) return;
    x.s0 = 0;
    x.s1 = p.a.seqs;
    x.k0 = x.k1 = 0;
  }
  const int k1 = x.k1;
  Rows it = x.it;
  it.h = __builtin_amdgcn_readfirstlane(it.h);
  if (prefix) it.r0 += 32 * wave;
  const bool live = it.r0 < it.rows;  // waves without rows only fetch
  Wave<DT, D> w;
  const bool some = x.k0 < k1, own = live && (!prefix || p.nos == 0);
  const int own_step = prefix ? p.nps : p.nos;
  F f;
  f.init(p);
  typename F::Half ha{}, hb{};
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_short*)smem;
  // 32 slots' places: K 0 to 3 (two tiles), V 4 to 7
  auto fetch_k = [&](const typename F::Half& h, int place) { f.rows(h.k, f.koff, lds + kRows * place); };
  auto fetch_v = [&](const typename F::Half& h, int place) { f.rows(h.v, f.voff, lds + kRows * place); };
  if (some) f.look(p, x.pages, x.k0, k1);
  load_q<DT, D>(p, it, w);
  if (some) {
    f.turn_to_next(p, it.h);
    f.take(p, x.pages, it.h, x.k0, k1, &ha, &hb);
    fetch_k(hb, 2);
    fetch_v(hb, 4);
    f.take(p, x.pages, it.h, x.k0, k1, &ha, &hb);
    fetch_k(ha, 0);
    fetch_v(ha, 5);
    fetch_k(hb, 1);
  }
  // What the own slots need is looked up while the first tiles are on their way.
  if (own) {
    const OwnRow r = own_row(p, it, x.s0, x.s1, part, own_step);
    const int page = own_total(r) > 0 ? own_look(p, r, 0, own_step).page : 0;
    if ((threadIdx.x & 63) < 32) {
      s_own[wave][threadIdx.x & 31] = r;
      s_page[wave][threadIdx.x & 31] = page;
    }
  }
  if (some) {
    wait_fetch();
    __syncthreads();
    f16v s[1], t[1];
    s8v kf[D / 16];
    float top = 0.f;
    if (live) {
      read_k<D>(smem + kRows, kf);  // its place becomes the second K tile's
      s[0] = f16v{};
#pragma unroll
      for (int i = 0; i < D / 16; ++i) s[0] = mfma<DT>(kf[i], w.q[i], s[0]);
      if (x.k0 + 32 > k1) mask_tile(s[0], x.k0, k1);
      top = top_of(s);
    }
    __syncthreads();
    // One step, on the tiles of parity b.
    auto step = [&](int k, int b) {
      const short* ks = smem + b * kRows;
      short* vs = smem + (2 + b) * kRows;
      if (k + kTile < k1) {
        fetch_v(hb, 6 - 2 * b);  // slots k + 64 ..
        f.take(p, x.pages, it.h, x.k0, k1, &ha, &hb);
        fetch_k(ha, 2 - 2 * b);  // slots k + 96 ..
        fetch_v(ha, 7 - 2 * b);
        fetch_k(hb, 3 - 2 * b);
      } else if (k + kTile > k1) {
        // values behind the end are cleared: a probability of zero must not meet an infinity
        for (int i = threadIdx.x; i < (k + kTile - k1) * (D / 8); i += NW * 64)
          *reinterpret_cast<u4*>(vs + (k1 - k) * D + 8 * i) = u4{0, 0, 0, 0};
        __syncthreads();
      }
      if (live) {
        read_k<D>(ks, kf);
        half_step<DT, D, true>(p, w, s, t, top, kf, vs, ks + 32 * D);
        if (k + 64 > k1) {
          mask_tile(t[0], k + 32, k1);
          top = top_of(t);
        }
        half_step<DT, D, false>(p, w, t, s, top, kf, vs + 32 * D, nullptr);
        if (k + 96 > k1) {
          mask_tile(s[0], k + 64, k1);
          top = top_of(s);
        }
      }
      wait_fetch();
      __syncthreads();
    };
    for (int k = x.k0; k < k1; k += 2 * kTile) {
      step(k, 0);
      if (k + kTile < k1) step(k + kTile, 1);
    }
  }
  if (!live) return;
  if (own)
    own_slots<DT, D>(p, w, s_own[wave][threadIdx.x & 31], s_page[wave][threadIdx.x & 31], it.h, own_step,
                     smem + wave * 64 * D);
  store_rows<DT, D>(p, it, w, prefix ? part : p.nps + part);
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
    // eight parts' loads at once; an empty part holds nothing, not zeros
    for (int i = 0; i < parts; i += 8) {
      f4 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        x[k] = *reinterpret_cast<const f4*>(p.part_o + (min(i + k, parts - 1) * rows + row) * D + 4 * min(l, D / 4 - 1));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float wgt = i < 32 ? __shfl(z0, i + k, 32) : __shfl(z1, i + k - 32, 32);
        if (i + k < parts && wgt != 0.f) acc += x[k] * wgt;
      }
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
  if (p.nps + p.nos == 1) return hipSuccess;
  const long long rows = (long long)p.a.tokens * p.a.q_heads;
  k_join<DT, D><<<(unsigned)std::min<long long>((rows + 7) / 8, 1 << 20), 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_prefix_attention(const PrefixArgs& a, const PrefixPlan& plan, char* ws, hipStream_t st) {
  PrefixDev p{};
  p.a = a;
  // A scale of 0 would turn a masked -infinity into NaN: the queries become 0
  // instead. The smallest others are subnormal here, at most 2^-150 off, which
  // moves a score (of products below 2^128) by at most 2^-22.
  p.zero = a.scale == 0.f;
  p.scale2 = p.zero ? 1.f : std::fabs(a.scale) * 1.4426950408889634f;
  p.q_sign = a.scale < 0.f ? 0x80008000u : 0u;
  p.m = a.q_heads / a.kv.heads;
  p.by_m = fast_div((uint32_t)p.m);
  p.nps = plan.nps;
  p.nos = plan.nos;
  p.prefix_tiles = (int)plan.prefix_tiles;
  p.prefix_blocks = (int)plan.prefix_blocks;
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
