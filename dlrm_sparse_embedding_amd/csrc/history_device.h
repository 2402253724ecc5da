// Device helpers of the attention of histories: the rows of a tile on their way
// into LDS and out of it, sequences' tiles, and the bias by relative position.
#pragma once

#include "attn_device.h"

namespace emb {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kHidden = -0x1p100f;  // entries of the bias from here down hide their distances

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

// Operand of rows row0 + lane % 32, contracted over their elements 16 i .. + 15.
template <int D>
__device__ __forceinline__ s8v row_operand(const short* tile, int row0, int i) {
  const int lane = threadIdx.x & 63, r = lane & 31;
  return *reinterpret_cast<const s8v*>(tile + (row0 + r) * D + 8 * ((2 * i + (lane >> 5)) ^ swizzle<D>(r)));
}
// Operand of the tile's columns 32 d + lane % 32, contracted over the 16 rows
// from row0 on, in the order that a product's elements 8 k .. 8 k + 7 have.
template <int D>
__device__ __forceinline__ s8v column_operand(const short* tile, int row0, int d, int lane) {
  const int q = lane & 15;
  const int r = 4 * (lane >> 5) + (q >> 2);
  const int c = (4 * d + 2 * ((lane >> 4) & 1) + ((q & 3) >> 1)) ^ swizzle<D>(r);
  const short* at = tile + (row0 + r) * D + 4 * (q & 1);
  const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(at + 8 * c));
  const s4v hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s4v*)(at + 8 * D + 8 * (c ^ 2)));  // swizzle(r + 8)
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

template <int D>
__device__ __forceinline__ s8v column_operand(const short* tile, int row0, int d) {
  return column_operand<D>(tile, row0, d, threadIdx.x & 63);
}

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
__device__ __forceinline__ void fetched() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ uint64_t uniform(uint64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)x), hi = __builtin_amdgcn_readfirstlane((int)(x >> 32));
  return (uint64_t)hi << 32 | lo;
}

// The fetches of a block of 256 threads: 64 rows are D / 32 for each thread.
template <int D>
struct RowFetch {
  static constexpr int kN = D / 32;
  int row[kN];        // of the tile
  uint32_t piece[kN];  // byte offset in it
  uint32_t wave_at;
  __device__ __forceinline__ RowFetch() {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int at = i * 256 + threadIdx.x;
      row[i] = at / (D / 8);
      piece[i] = 16 * ((at % (D / 8)) ^ swizzle<D>(row[i]));
    }
    wave_at = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
  }
  // Rows of `stride` bytes from `base` (the tile's first row) into `tile`; rows
  // beyond `last` repeat it.
  __device__ __forceinline__ void rows(uint64_t base, uint32_t stride, int last, uint32_t tile) const {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      fetch_to_lds(base, (uint32_t)min(row[i], last) * stride + piece[i], tile + wave_at + 4096 * i);
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
__device__ __forceinline__ float bias_log2(float b) { return b <= kHidden ? kNegInf : b * kLog2e; }

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
__device__ __forceinline__ Biases biases_of(const HistoryView& h, const BiasLds& s, int delta_max, float* win) {
  Biases b;
  const int last = h.buckets.n - 1, bound = h.buckets.first[last];
  const int delta_min = delta_max - 62;
  b.far = delta_min >= bound || (!h.causal && delta_max <= -bound);
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
// Whether any of the wave's 32 rows of D elements at v holds an infinity or NaN.
template <int DT, int D>
__device__ __forceinline__ bool any_special(const short* v) {
  typedef unsigned short us8 __attribute__((ext_vector_type(8)));
  constexpr unsigned short top = DT == EMB_BF16 ? 0x7f80 : 0x7c00;
  unsigned m = 0;
#pragma unroll
  for (int i = 0; i < 32 * D / 512; ++i) {
    const us8 x = *reinterpret_cast<const us8*>(v + 8 * (i * 64 + (threadIdx.x & 63)));
#pragma unroll
    for (int j = 0; j < 8; ++j) m |= (x[j] & top) == top ? 1u : 0u;
  }
  return __ballot(m != 0) != 0;
}

// acc[d] += (columns of 32 rows of the tile, from row0 on) times w, for a tile in
// which not every column of w sees every row: those that it does not see have a
// weight of 0, but an infinity or NaN there would still reach it. Column c sees
// the rows [lo, hi) (the lane's own), counted from row0. Rare: only tiles with
// such values come here. One product for each of the bounds, with the rows
// beyond it cleared, of which each column keeps its own.
template <int DT, int D>
__device__ __forceinline__ void guarded_product(f16v (&acc)[D / 32], const short* tile, int row0, const s8v (&w)[2],
                                                int lo, int hi) {
#pragma unroll 1
  for (int a = 0; a < 32; ++a) {
    // What is worked out from the lane stays in here: held outside, for this rare
    // path, it would take registers from the common one.
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    const int l = __builtin_amdgcn_readlane(lo, a), u = __builtin_amdgcn_readlane(hi, a);
    const bool mine = (lane & 31) == a;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) {
      f16v o = acc[d];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        s8v x = column_operand<D>(tile, row0 + 16 * k, d, lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = 16 * k + 8 * (j / 4) + 4 * (lane >> 5) + j % 4;
          x[j] = r >= l && r < u ? x[j] : (short)0;
        }
        o = mfma<DT>(x, w[k], o);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[d][i] = mine ? o[i] : acc[d][i];
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// Packs the elements of a product, times `by`, for the next one.
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

// The operands of row `row` (one a lane column) of a heads operand.
template <int D>
__device__ __forceinline__ void load_operands(const Heads& x, long long token, int head, s8v (&f)[D / 16]) {
  const short* src = reinterpret_cast<const short*>(x.p) + token * x.ts + head * x.hs + 8 * ((threadIdx.x & 63) >> 5);
#pragma unroll
  for (int i = 0; i < D / 16; ++i) f[i] = *reinterpret_cast<const s8v*>(src + 16 * i);
}

}  // namespace emb
