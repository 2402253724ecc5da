// Declarations shared by the sequence operators' kernels and their C-ABI
// host layer (emb_seq.cpp). Not part of the public interface.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "emb.h"

namespace emb {

// The error reporting of the C ABI (emb_api.cpp), per thread.
int fail(int code, const char* fmt, ...);
int ok();
int hip_fail(hipError_t e, const char* what);

// Frequencies of a rotation. turn[i] is pair i's angle per position as a
// fraction of a whole turn, in units of 2^-64: position * turn[i] modulo 2^64
// is the angle, whole turns dropped, with no rounding but the frequency's own.
struct RotTable {
  uint64_t turn[EMB_MAX_ROT / 2];
  float mag;
  int32_t rot;     // 0: no rotation
  int32_t layout;  // EMB_ROT_*
};

// [tokens][heads][dim] in memory; strides in elements.
struct Heads {
  const void* p;
  long long ts, hs;
  int n;
};

// n / d for 0 <= n < 2^31 as a product and a shift: with s = ceil(log2 d) and
// mul = floor(2^(31+s) / d) + 1, n * mul >> (31 + s) is exact.
struct FastDiv {
  uint32_t mul, shift, d;
};
FastDiv fast_div(uint32_t d);

// Device view of a paged cache.
struct KvView {
  char* k;
  char* v;
  long long kps, kss, khs, vps, vss, vhs;  // strides in elements
  int pages, page, heads, dim, dtype;
  FastDiv by_page;
  int* error;  // may be null
};

// bits of the cache's error flag
constexpr int kKvBadPage = 1;
constexpr int kKvBadOffsets = 2;

// ---- rotary positions and head norms (k_rotary.hip) ----
// y = rotate(x) or, with norm, rotate(x * r * w); both operands in one launch.
struct NormRotaryArgs {
  const void* positions;
  int itype;
  long long tokens;
  int dtype, dim;
  Heads q, qo, k, ko;  // *o.p is written
  int inverse, norm;
  const float *wq, *wk;
  float eps;
};
hipError_t launch_norm_rotary(const NormRotaryArgs& a, const RotTable& rot, hipStream_t st);

struct NormRotaryBackArgs {
  const void* positions;
  int itype;
  long long tokens;
  int dtype, dim;
  Heads q, dyq, dq, k, dyk, dk;
  const float *wq, *wk;
  float eps;
  float* part;  // [blocks][2][dim]
  float *dwq, *dwk;
};
int norm_rotary_back_blocks(long long tokens, int hq, int hk, int dim);
hipError_t launch_norm_rotary_back(const NormRotaryBackArgs& a, const RotTable& rot, hipStream_t st);

struct AppendArgs {
  KvView kv;
  long long tokens;
  Heads k, v;
  const int* offsets;  // null: one token per sequence
  int seqs;
  const int* lens;
  const int* table;
  int width;
  const void* positions;  // null: the slot
  int itype;
  int norm;
  const float* wk;
  float eps;
};
hipError_t launch_kv_append(const AppendArgs& a, const RotTable& rot, hipStream_t st);

// ---- attention over a shared prefix and the own sequence (k_prefix.hip) ----
struct PrefixArgs {
  KvView kv;
  int tokens, q_heads;
  Heads q, out;
  float scale;
  const int* offsets;
  int seqs;
  const int* lens;
  const int* table;
  int width;
  const int* group_offsets;
  int groups;
  const int* prefix_lens;
  const int* prefix_table;
  int pwidth;
  float* lse;  // may be null
};

// How the keys are split, the grid, and what the workspace holds: `nps` parts
// of a prefix and `nos` parts of an own sequence, each a partial output with
// its log-sum per (token, query head). The host does not know where groups
// and sequences begin, so tiles are counted by an upper bound: tiles of R rows
// of group (sequence) i are numbered from i + floor(first row / R).
struct PrefixPlan {
  int nps, nos;
  bool wide;   // prefix tiles of 128 rows that share their keys in LDS, else 32
  long long prefix_tiles, prefix_blocks, own_tiles, own_blocks;
  size_t o_off;     // partial outputs fp32 [nps + nos][tokens][q_heads][dim]
  size_t lse_off;   // fp32 [nps + nos][tokens][q_heads]
  size_t bytes;
};
PrefixPlan prefix_plan(const KvView& kv, long long tokens, int q_heads, int groups, int pwidth,
                       int width);
hipError_t launch_prefix_attention(const PrefixArgs& a, const PrefixPlan& p, char* ws, hipStream_t st);

}  // namespace emb
