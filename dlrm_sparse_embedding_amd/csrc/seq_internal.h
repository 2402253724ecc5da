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

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline int esize(int dtype) { return dtype == EMB_F32 ? 4 : 2; }

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

// Checks of arguments (emb_seq.cpp); EMB_OK or the code of a reported failure.
int check_dtype(int dtype);
int check_heads(const char* name, const Heads& h, int dtype);
int check_out(const char* name, const Heads& h, long long tokens, int dim, int dtype);
int check_norm(const char* name, const float* w, float eps);

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

// ---- layer norm and dropout (k_rows.hip) ----
// [rows][dim] in memory; stride in elements.
struct Rows2D {
  const void* p;
  long long stride;
  int dtype;
};

struct LayerNormArgs {
  long long rows;
  int dim;
  Rows2D x, y;  // y.p is written
  const float *w, *b;
  float eps;
};
hipError_t launch_layer_norm(const LayerNormArgs& a, hipStream_t st);

struct LayerNormBackArgs {
  long long rows;
  int dim;
  Rows2D x, dy, dx;
  const float* w;
  float eps;
  float* part;  // [blocks][2][dim]
  float *dw, *db;
};
int layer_norm_back_blocks(long long rows);  // upper bound
hipError_t launch_layer_norm_back(const LayerNormBackArgs& a, hipStream_t st);

struct DropoutArgs {
  long long rows;
  int dim;
  Rows2D x, res, y;  // res.p may be null
  uint64_t threshold;  // t of p = t / 2^32, at most 2^32
  float scale;         // 1 / (1 - p)
  uint64_t seed;
  const long long* step;  // may be null
};
hipError_t launch_dropout(const DropoutArgs& a, hipStream_t st);

// ---- attention of histories (k_history.hip, k_history_back.hip, k_history_step.hip) ----
// Buckets of distances d >= 0: d below `exact`, then those that start at
// first[exact] = exact, .., first[buckets - 1]; first[buckets] is 2^31 - 1.
struct Buckets {
  int n, exact;             // n = 0: no bias
  int first[EMB_MAX_BUCKETS + 1];
  float log2_exact, slope;  // the bucket is exact + (log2 d - log2_exact) * slope, to within one
};

struct HistoryView {
  int q_heads, kv_heads, dim, dtype, causal;
  float scale;
  Buckets buckets;
  int* error;  // may be null
};

struct HistoryArgs {
  HistoryView h;
  int tokens, seqs;
  Heads q, k, v, out;  // out.p is written by the forward
  const int* offsets;
  const float* bias;  // null where there are no buckets
  float* lse;         // may be null in the forward
};
hipError_t launch_history(const HistoryArgs& a, hipStream_t st);

struct HistoryBackArgs {
  HistoryArgs f;
  Heads dout, dq, dk, dv;
  float* dbias;  // may be null
  float* rows;   // workspace: [2][q_heads][tokens]: sums P dP, z in log2 units
  float* part;   // workspace: [blocks][rows of the bias] partial sums of dbias
};
// What the workspace holds (bytes): the rows' sums, then the partial sums.
struct HistoryBackPlan {
  size_t part_off, bytes;
};
HistoryBackPlan history_back_plan(const HistoryView& h, long long tokens, int seqs);
hipError_t launch_history_back(const HistoryBackArgs& a, hipStream_t st);

struct HistoryStepArgs {
  HistoryView h;
  KvView kv;
  int seqs;
  Heads q, out;
  const int* lens;
  const int* table;
  int width;
  const float* bias;
  float* lse;
  int parts;
  float* part_o;    // [parts][seqs][q_heads][dim]
  float* part_lse;  // [parts][seqs][q_heads]
};
int history_step_parts(const HistoryView& h, const KvView& kv, int seqs, int width);
hipError_t launch_history_step(const HistoryStepArgs& a, hipStream_t st);

}  // namespace emb

struct emb_kv {
  emb::KvView v;
};

struct emb_history {
  emb::HistoryView v;
};
