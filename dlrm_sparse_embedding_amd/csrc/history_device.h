// Device helpers of the attention of histories: the rows of a tile on their way
// into LDS and out of it, sequences' tiles, and the bias by relative position.
#pragma once

#include "attn_device.h"

namespace emb {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---- tiles in LDS -------------------------------------------------------------
// 64 rows of D elements without padding; 16-byte piece c of row r lies at c ^
// swizzle(r). Tiles are read in two ways, whole rows (16 bytes of 16 rows at
// once) and transposed (8 bytes of 4 neighbouring rows): with this swizzle both
// find different banks, so one tile serves both.
constexpr int kTile = 64;

template <int D>
__device__ __forceinline__ int swizzle(int r) {
  if constexpr (D == 128) return 4 * (r & 3) ^ ((r >> 2) & 3);
  else if constexpr (D == 64) return 4 * ((r >> 1) & 1) | ((r >> 2) & 3);
  else return (r >> 2) & 3;
}

// Where a lane reads in a tile, as byte offsets: of its row's operands and of its
// columns' two halves. The 16-byte pieces of a row are a power of two (D = 64,
// 128), so that an operand's piece is one exclusive or away; for D = 96 their
// lowest two bits are swizzled and two offsets are kept.
template <int D>
struct TileLane {
  uint32_t row[D == 96 ? 2 : 1], col[2];
  __device__ __forceinline__ TileLane() : TileLane(threadIdx.x & 63) {}
  __device__ __forceinline__ explicit TileLane(int lane) {
    const int r = lane & 31, h = lane >> 5;
    row[0] = 2 * D * r + 16 * (h ^ swizzle<D>(r));
    if constexpr (D == 96) row[1] = 2 * D * r + 16 * ((2 + h) ^ swizzle<D>(r));
    const int q = lane & 15, cr = 4 * h + (q >> 2);
    const int c = (2 * ((lane >> 4) & 1) + ((q & 3) >> 1)) ^ swizzle<D>(cr);
    col[0] = 2 * D * cr + 8 * (q & 1) + 16 * c;
    col[1] = 2 * D * (cr + 8) + 8 * (q & 1) + 16 * (c ^ 2);  // swizzle(r + 8) = swizzle(r) ^ 2
  }
  // Offsets that the compiler takes as new: what is worked out from them is not
  // held in registers beyond this point.
  __device__ __forceinline__ TileLane fresh() const {
    TileLane t = *this;
#pragma unroll
    for (uint32_t& x : t.row) asm volatile("" : "+v"(x));
    asm volatile("" : "+v"(t.col[0]), "+v"(t.col[1]));
    return t;
  }
  // Operand of the tile's rows row0 + lane % 32, contracted over their elements 16 i .. + 15.
  __device__ __forceinline__ s8v rows(const short* tile, int row0, int i) const {
    const uint32_t at = D == 96 ? row[(i & 1) * (D == 96)] + 64 * (i / 2) : row[0] ^ (32 * i);
    return *reinterpret_cast<const s8v*>(reinterpret_cast<const char*>(tile) + 2 * D * row0 + at);
  }
  // Operand of the tile's columns 32 d + lane % 32, contracted over the 16 rows
  // from row0 on, in the order that a product's elements 8 k .. 8 k + 7 have.
  __device__ __forceinline__ s8v columns(const short* tile, int row0, int d) const {
    const uint32_t a = D == 96 ? col[0] + 64 * d : col[0] ^ (64 * d), b = D == 96 ? col[1] + 64 * d : col[1] ^ (64 * d);
    const char* at = reinterpret_cast<const char*>(tile) + 2 * D * row0;
    const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(at + a));
    const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(at + b));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  }
};

typedef __attribute__((address_space(3))) short lds_elem;

// 16 bytes for each lane from base + off into LDS at `at` + 16 * lane. The
// compiler does not see the transfer: the caller waits (fetched) and passes a
// barrier before anyone reads. It does not see the instruction's hazards either:
// a base that a vector instruction wrote would have to be five wait states old,
// so a scalar one copies it, and that copy is the wait state which m0 needs.
__device__ __forceinline__ void fetch_to_lds(uint64_t base, uint32_t off, uint32_t at) {
  uint64_t from;
  asm volatile("s_mov_b64 %0, %3\n\tglobal_load_lds_dwordx4 %2, %0"
               : "=&s"(from)
               : "{m0}"(at), "v"(off), "s"(base)
               : "memory");
}
// The same with 4 bytes a lane.
__device__ __forceinline__ void fetch_word_to_lds(uint64_t base, uint32_t off, uint32_t at) {
  uint64_t from;
  asm volatile("s_mov_b64 %0, %3\n\tglobal_load_lds_dword %2, %0"
               : "=&s"(from)
               : "{m0}"(at), "v"(off), "s"(base)
               : "memory");
}
typedef __attribute__((address_space(3))) float lds_word;
__device__ __forceinline__ void fetched() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint64_t uniform(uint64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)x), hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
  return (uint64_t)hi << 32 | lo;
}

// The fetches of a block of 256 threads: 64 rows are D / 32 for each thread.
template <int D>
struct RowFetch {
  static constexpr int kN = D / 32, kKept = D == 96 ? kN : 1;
  int row[kKept];        // of the tile
  uint32_t piece[kKept];  // byte offset in it
  uint32_t wave_at;
  __device__ __forceinline__ RowFetch() {
#pragma unroll
    for (int i = 0; i < kKept; ++i) {
      const int at = i * 256 + threadIdx.x;
      row[i] = at / (D / 8);
      piece[i] = 16 * ((at % (D / 8)) ^ swizzle<D>(row[i]));
    }
    wave_at = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
  }
  // 64 rows of `stride` bytes, `from` of those at `base` on, into `tile`; rows
  // beyond the `last` of them repeat it. Where the rows' pieces are a power of two, a thread's
  // rows are 2048 / D apart and swizzle alike.
  __device__ __forceinline__ void rows(uint64_t base, uint32_t stride, int from, int last, uint32_t tile) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int r = kKept == 1 ? row[0] + 2048 / D * i : row[i];
      fetch_to_lds(base, (uint32_t)min(r + from, last) * stride + piece[kKept == 1 ? 0 : i], tile + wave_at + 4096 * i);
    }
  }
};

// ---- sequences' tiles ----------------------------------------------------------
// Tiles of R rows: tile i of the sequence whose tiles start at b + offsets[b] /
// R, which counts more tiles than there are, without the lengths.
struct SeqTile {
  int b, first, len;  // sequence, its first token, its tokens
  int r0;             // first row of the tile in it; at least len where there is none
};
__device__ __forceinline__ int first_of(const HistoryArgs& a, int b) { return min(max(a.offsets[b], 0), a.tokens); }
__device__ __forceinline__ SeqTile seq_tile(const HistoryArgs& a, int tile, int R) {
  SeqTile t;
  t.b = wave_find(a.seqs, tile, [&](int i) { return i + first_of(a, i) / R; });
  t.first = __builtin_amdgcn_readfirstlane(first_of(a, t.b));
  t.len = __builtin_amdgcn_readfirstlane(first_of(a, t.b + 1)) - t.first;
  t.r0 = (tile - (t.b + t.first / R)) * R;
  if (t.r0 < 0) t.r0 = t.len;
  return t;
}
// Heads and tiles of a grid of heads * tiles blocks, heads fastest. Blocks are
// dealt to the 8 XCDs in turn; where the heads can be, they are dealt so that an
// XCD has neighbouring ones, which share their key head, and with it the L2.
__device__ __forceinline__ void head_and_tile(int block, int heads, FastDiv by_heads, int* head, int* tile) {
  *tile = div_by(by_heads, block);
  const int h = block - *tile * heads;
  *head = heads % 8 == 0 ? (h & 7) * (heads >> 3) + (h >> 3) : h;
}
inline long long seq_tiles(long long tokens, int seqs, int R) { return seqs + tokens / R; }

// ---- the bias --------------------------------------------------------------------
// Bucket of a distance d >= 0 from the logarithm, which is off by one at most,
// and the buckets' bounds.
__device__ __forceinline__ int bucket_of(const Buckets& k, const int* first, int d) {
  const int guess = (int)((__log2f((float)max(d, 1)) - k.log2_exact) * k.slope) + k.exact;
  int g = min(max(guess, k.exact), k.n - 1);
  g += d >= first[g + 1] ? 1 : 0;
  g -= d < first[g] ? 1 : 0;
  return d < k.exact ? min(d, k.n - 1) : g;
}
// Row of the bias for a query `delta` places behind its key. Neighbouring deltas
// have one row or rows of their own: causal ones below 0, which nobody sees, have
// that of 0.
__device__ __forceinline__ int bias_row(const HistoryView& h, const int* first, int delta) {
  const int d = h.causal ? max(delta, 0) : delta;
  const int g = bucket_of(h.buckets, first, d < 0 ? -d : d);
  return d < 0 ? g + h.buckets.n : g;
}
// A bias as the kernels use it: in units of log2, minus infinity where it hides.
__device__ __forceinline__ float bias_log2(float b) { return b <= EMB_HIDDEN_BIAS ? kNegInf : b * kLog2e; }

// A block's copy of the bounds and of one head's bias.
struct BiasLds {
  int first[EMB_MAX_BUCKETS + 1];
  float value[2 * EMB_MAX_BUCKETS];
};
__device__ __forceinline__ void stage_bounds(const HistoryView& h, BiasLds& s) {
  for (int i = threadIdx.x; i <= h.buckets.n; i += blockDim.x) s.first[i] = h.buckets.first[i];
}
__device__ __forceinline__ void stage_bias(const HistoryArgs& a, int head, BiasLds& s) {
  const int rows = a.h.buckets.n * (a.h.causal ? 1 : 2);
  for (int i = threadIdx.x; i < rows; i += blockDim.x) s.value[i] = bias_log2(a.bias[(long long)i * a.h.q_heads + head]);
}

// What a wave knows of the 63 distances between its 32 rows of one side and 32
// of the other: where all of them are in one last bucket (`far`), its value;
// otherwise lane x < 63 has the row of distance delta_max - x and `win[x]` its
// bias.
struct Biases {
  bool far;
  float value;  // of the far bucket
  int row;      // uniform where far, else the lane's
};
// delta_max: the largest distance (query place minus key place).
__device__ __forceinline__ bool all_far(const HistoryView& h, int delta_max, int delta_min) {
  const int bound = h.buckets.first[h.buckets.n - 1];
  return delta_min >= bound || (!h.causal && delta_max <= -bound);
}
// near: the window also where all are far.
__device__ __forceinline__ Biases biases_of(const HistoryView& h, const BiasLds& s, int delta_max, float* win,
                                            bool near = false) {
  Biases b;
  const int last = h.buckets.n - 1, bound = h.buckets.first[last];
  const int delta_min = delta_max - 62;
  b.far = !near && all_far(h, delta_max, delta_min);
  if (b.far) {
    b.row = delta_min >= bound ? last : last + h.buckets.n;
    b.value = s.value[b.row];
  } else {
    const int lane = threadIdx.x & 63;
    b.row = bias_row(h, s.first, delta_max - min(lane, 62));
    b.value = 0.f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // earlier reads of win are over
    win[lane] = s.value[b.row];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  return b;
}

// ---- values that are not numbers ----------------------------------------------
// A product over a tile's rows gives rows that a column does not see a weight of
// 0, but an infinity or NaN there would still reach it. Only tiles on the diagonal
// of causal calls and those with the sequence's end have such rows; where one of
// them holds such values, which is rare, its block takes them out of LDS between
// the tile's scores, which still need them, and its product, and (for values whose
// weights are positive) notes where they were: Marks.

constexpr int kNoMark = 0x7fffffff;

// For each of D elements the row nearest to those that do not see it that holds
// +infinity, -infinity, NaN there: the first (sign 1) or the last (sign -1; all
// rows times the sign).
template <int D>
struct Marks {
  int at[3][D];
  __device__ __forceinline__ void clear() {
    for (int i = threadIdx.x; i < 3 * D; i += blockDim.x) (&at[0][0])[i] = kNoMark;
  }
};

// Whether the block's `rows` rows of D elements at `tile` hold infinities or NaN.
// Contains a barrier.
template <int DT, int D>
__device__ __forceinline__ bool any_special(const short* tile, int rows) {
  constexpr uint32_t top = DT == EMB_BF16 ? 0x7f80u : 0x7c00u;
  int found = 0;
  for (int i = threadIdx.x; i < rows * (D / 8); i += 256) {
    const u4 x = *reinterpret_cast<const u4*>(tile + 8 * i);
#pragma unroll
    for (int j = 0; j < 4; ++j) found |= (x[j] & top) == top || (x[j] >> 16 & top) == top;
  }
  return __syncthreads_or(found) != 0;
}

// Takes them out of 32 rows, the first of which is row `first` of `len` of its
// sequence: rows behind the end become zeros; of the others, where `inside`,
// infinities and NaN, which go into `marks` (may be null) as rows times `sign`.
template <int DT, int D>
__device__ __forceinline__ void clear_special(short* tile, int first, int len, bool inside, Marks<D>* marks, int sign) {
  constexpr uint32_t top = DT == EMB_BF16 ? 0x7f80u : 0x7c00u;
  for (int i = threadIdx.x; i < 32 * (D / 8); i += 256) {
    const int r = i / (D / 8), c = 8 * (i % (D / 8) ^ swizzle<D>(r));
    short* at = tile + 8 * i;
    if (first + r >= len) {
      *reinterpret_cast<s8v*>(at) = s8v{};
    } else if (inside) {
      for (int j = 0; j < 8; ++j) {
        const uint32_t x = (uint16_t)at[j];
        if ((x & top) != top) continue;
        at[j] = 0;
        const int kind = (x & 0x7fffu) > top ? 2 : (int)(x >> 15);
        if (marks) atomicMin(&marks->at[kind][c + j], sign * (first + r));
      }
    }
  }
}

// What the lane's column, at `place` times the sign, sees of the marks, added to
// its sums.
template <int D>
__device__ __forceinline__ void add_marks(f16v (&acc)[D / 32], const Marks<D>& marks, int place) {
  const int h4 = 4 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int c = 32 * d + 8 * (i / 4) + h4 + i % 4;
      const bool u = place >= marks.at[0][c], v = place >= marks.at[1][c], n = place >= marks.at[2][c] || (u && v);
      acc[d][i] += n ? __builtin_nanf("") : u ? -kNegInf : v ? kNegInf : 0.f;
    }
}

// The operands of 32 rows of a tile, read together ahead of the products that use
// them: left to the compiler, each product waits for its own read.
template <int D>
struct RowOps {
  s8v x[D / 16];
  __device__ __forceinline__ void read(const TileLane<D>& at, const short* tile) {
#pragma unroll
    for (int i = 0; i < D / 16; ++i) x[i] = at.rows(tile, 0, i);
  }
  template <int DT>
  __device__ __forceinline__ f16v times(const s8v (&w)[D / 16]) const {
    f16v s{};
#pragma unroll
    for (int i = 0; i < D / 16; ++i) s = mfma<DT>(x[i], w[i], s);
    return s;
  }
};
template <int D>
struct ColumnOps {
  s8v x[2][D / 32];
  __device__ __forceinline__ void read(const TileLane<D>& at, const short* tile) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int d = 0; d < D / 32; ++d) x[k][d] = at.columns(tile, 16 * k, d);
  }
  template <int DT>
  __device__ __forceinline__ void times(f16v (&acc)[D / 32], const s8v (&w)[2]) const {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int d = 0; d < D / 32; ++d) acc[d] = mfma<DT>(x[k][d], w[k], acc[d]);
  }
};
// Nothing moves across it.
__device__ __forceinline__ void stage() { __builtin_amdgcn_sched_barrier(0); }
// Asks for N products with VALU vector instructions behind each of them.
template <int N, int VALU>
__device__ __forceinline__ void interleave() {
  if constexpr (N > 0) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
    interleave<N - 1, VALU>();
  }
}

// acc[d] += (columns of the 32 rows at `tile`) times w.
template <int DT, int D>
__device__ __forceinline__ void add_product(f16v (&acc)[D / 32], const TileLane<D>& at, const short* tile,
                                            const s8v (&w)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int d = 0; d < D / 32; ++d) acc[d] = mfma<DT>(at.columns(tile, 16 * k, d), w[k], acc[d]);
}

// Which of a product's 32 rows are in [lo, hi): bit 8 (i / 4) + i % 4 for the
// lane's element i. One register for all of them, where comparisons would hold
// a mask each.
__device__ __forceinline__ uint32_t row_bits(int lo, int hi) {
  const int l = min(max(lo, 0), 32), u = min(max(hi, 0), 32);
  const uint64_t bits = ((1ull << u) - 1) & ~((1ull << l) - 1);
  return (uint32_t)bits >> 4 * ((threadIdx.x & 63) >> 5);
}
// x where element i's bit is set, else 0 (whatever x is).
__device__ __forceinline__ float where_bit(uint32_t bits, int i, float x) {
  const int mask = (int)(bits << (31 - (8 * (i / 4) + i % 4))) >> 31;
  return __uint_as_float(__float_as_uint(x) & (uint32_t)mask);
}

// Packs the elements of a product for the next one.
template <int DT>
__device__ __forceinline__ void pack_tile(const f16v& x, s8v (&w)[2]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
    w[k] = __builtin_bit_cast(s8v, u4{pack2<DT>(x[8 * k], x[8 * k + 1]), pack2<DT>(x[8 * k + 2], x[8 * k + 3]),
                                      pack2<DT>(x[8 * k + 4], x[8 * k + 5]), pack2<DT>(x[8 * k + 6], x[8 * k + 7])});
}

// Stores 32 columns of a product over D rows as rows of memory: lane's column to
// `dst` (its row's first element + 8 * (lane / 32)), times `by`. Lanes l and l +
// 32 hold 4 of every 8; they trade halves so that one stores elements 16 i .. + 7
// and the other the next 8.
template <int DT, int D>
__device__ __forceinline__ void store_columns(short* dst, const f16v (&o)[D / 32], float by, bool store) {
  typedef unsigned u2v __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f16v& x = o[d];
      const u2v lo = __builtin_amdgcn_permlane32_swap(pack2<DT>(x[8 * i] * by, x[8 * i + 1] * by),
                                                      pack2<DT>(x[8 * i + 4] * by, x[8 * i + 5] * by), false, false);
      const u2v hi = __builtin_amdgcn_permlane32_swap(pack2<DT>(x[8 * i + 2] * by, x[8 * i + 3] * by),
                                                      pack2<DT>(x[8 * i + 6] * by, x[8 * i + 7] * by), false, false);
      if (store) *reinterpret_cast<u4*>(dst + 32 * d + 16 * i) = u4{lo.x, hi.x, lo.y, hi.y};
    }
}

// The operands of a token (one a lane column). They are waited for here: left to
// their first use, inside the loop over the tiles, the wait would be repeated there
// and take in the tile that has just been asked for.
template <int D>
__device__ __forceinline__ void load_operands(const Heads& x, long long token, int head, s8v (&f)[D / 16]) {
  const short* src = reinterpret_cast<const short*>(x.p) + token * x.ts + head * x.hs + 8 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) f[i] = *reinterpret_cast<const s8v*>(src + 16 * i);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) asm volatile("" : "+v"(f[i]));
}

}  // namespace emb
