// C-ABI host layer of the history layer (layer norm, dropout, attention of
// histories): argument validation and workspace sizes. No C++ exception
// crosses the ABI.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <new>

#include "emb.h"
#include "seq_internal.h"

using namespace emb;

namespace {

int check_rows_sizes(int64_t rows, int32_t dim, int64_t max_dim) {
  if (rows < 0 || rows >= (1ll << 31)) return fail(EMB_E_INVAL, "rows %lld not in [0, 2^31)", (long long)rows);
  if (dim < 1 || dim > max_dim) return fail(EMB_E_INVAL, "dim %d not in [1, %lld]", dim, (long long)max_dim);
  return EMB_OK;
}

int check_rows(const char* name, const Rows2D& r) {
  if (!r.p) return fail(EMB_E_INVAL, "%s is NULL", name);
  if (!aligned(r.p, (size_t)esize(r.dtype))) return fail(EMB_E_INVAL, "%s is not aligned to its elements", name);
  if (r.stride < 0) return fail(EMB_E_INVAL, "%s has a negative stride", name);
  return EMB_OK;
}

int check_rows_out(const char* name, const Rows2D& r, int64_t rows, int32_t dim) {
  if (int rc = check_rows(name, r)) return rc;
  if (rows > 1 && r.stride < dim) return fail(EMB_E_INVAL, "%s: rows of stride %lld overlap", name, r.stride);
  return EMB_OK;
}

// Overlap of two operands is only allowed as the very same one.
int check_same(const char* in_name, const Rows2D& in, const char* out_name, const Rows2D& out) {
  if (in.p == out.p && (in.stride != out.stride || in.dtype != out.dtype))
    return fail(EMB_E_INVAL, "%s is %s with another stride or type", out_name, in_name);
  return EMB_OK;
}

int check_types(int x_dtype, int y_dtype) {
  if (int rc = check_dtype(x_dtype)) return rc;
  if (int rc = check_dtype(y_dtype)) return rc;
  if (x_dtype != y_dtype && x_dtype != EMB_F32)
    return fail(EMB_E_DTYPE, "y_dtype %d with x_dtype %d: the same, or 16-bit rows of fp32 ones", y_dtype, x_dtype);
  return EMB_OK;
}

// A number of up to 130 x 32 bits, for products of powers.
struct Wide {
  uint32_t w[130] = {1};
  int n = 1;
  void times(uint32_t x) {
    uint64_t carry = 0;
    for (int i = 0; i < n; ++i) {
      carry += (uint64_t)w[i] * x;
      w[i] = (uint32_t)carry;
      carry >>= 32;
    }
    if (carry && n < 130) w[n++] = (uint32_t)carry;
  }
  bool operator>=(const Wide& o) const {
    if (n != o.n) return n > o.n;
    for (int i = n - 1; i >= 0; --i)
      if (w[i] != o.w[i]) return w[i] > o.w[i];
    return true;
  }
};

// Whether d >= exact (far / exact)^(k / n), that is d^n >= exact^(n - k) far^k:
// factors below 2^31, n <= 127, so that either side has at most 3937 bits.
bool reaches(uint32_t d, uint32_t exact, uint32_t far, int k, int n) {
  Wide a, b;
  for (int i = 0; i < n; ++i) {
    a.times(d);
    b.times(i < k ? far : exact);
  }
  return a >= b;
}

Buckets make_buckets(const emb_history_desc& d) {
  Buckets b{};
  b.n = d.buckets;
  b.exact = d.exact;
  const int n = d.buckets - d.exact;
  for (int i = 0; i < d.buckets; ++i) {
    const int k = i - d.exact;
    uint32_t at = (uint32_t)i;
    if (k > 0) {
      const long double x = d.exact * powl((long double)d.far / d.exact, (long double)k / n);
      at = (uint32_t)x;
      while (!reaches(at, (uint32_t)d.exact, (uint32_t)d.far, k, n)) ++at;
      while (reaches(at - 1, (uint32_t)d.exact, (uint32_t)d.far, k, n)) --at;
    }
    b.first[i] = (int)at;
  }
  b.first[d.buckets] = 0x7fffffff;
  if (n > 0) {
    b.log2_exact = (float)std::log2((double)d.exact);
    b.slope = (float)(n / std::log2((double)d.far / d.exact));
  }
  return b;
}

// A launch has less than 2^32 threads, that is 2^24 blocks of 256.
constexpr long long kMaxBlocks = 1ll << 24;

bool too_many(const HistoryView& h, long long tokens, int seqs) {
  return (seqs + tokens / 64) * h.q_heads >= kMaxBlocks || tokens * h.q_heads >= (1ll << 31);
}

// Sequences of a call on ragged operands.
int check_ragged(const emb_history* h, int64_t tokens, const int32_t* offsets, int32_t seqs, const float* bias) {
  if (!h) return fail(EMB_E_INVAL, "history is NULL");
  if (tokens < 0 || tokens >= (1ll << 24)) return fail(EMB_E_INVAL, "tokens %lld not in [0, 2^24)", (long long)tokens);
  if (seqs < 0 || seqs >= (1 << 24)) return fail(EMB_E_INVAL, "seqs %d not in [0, 2^24)", seqs);
  if (seqs == 0 && tokens > 0) return fail(EMB_E_INVAL, "tokens without a sequence");
  if (too_many(h->v, tokens, seqs)) return fail(EMB_E_INVAL, "too many tokens or sequences for one call");
  if (h->v.buckets.n > 0 && (!bias || !aligned(bias, 4))) return fail(EMB_E_INVAL, "bias is NULL or misaligned");
  if (h->v.buckets.n == 0 && bias) return fail(EMB_E_INVAL, "bias without buckets");
  if (tokens > 0 && (!offsets || !aligned(offsets, 4))) return fail(EMB_E_INVAL, "offsets are NULL or misaligned");
  return EMB_OK;
}

// A heads operand of 16-byte accesses. Rows of a tile are addressed by 32-bit offsets.
int check_wide(const char* name, const Heads& x, long long tokens, const HistoryView& h, bool written) {
  if (int rc = written ? check_out(name, x, tokens, h.dim, h.dtype) : check_heads(name, x, h.dtype)) return rc;
  if (!aligned(x.p, 16) || x.ts % 8 != 0 || x.hs % 8 != 0)
    return fail(EMB_E_INVAL, "%s needs 16-byte alignment and strides of multiples of 16 bytes", name);
  if (x.ts >= (1ll << 24)) return fail(EMB_E_INVAL, "%s: a token stride of 2^24 elements or more", name);
  return EMB_OK;
}

// A written operand that starts where one that other blocks read does.
int check_apart(const char* name, const Heads& out, std::initializer_list<Heads> others) {
  for (const Heads& o : others)
    if (o.p == out.p) return fail(EMB_E_INVAL, "%s is another operand's memory", name);
  return EMB_OK;
}

// out may be q with the same strides: a block reads its queries before it writes their rows, and no other block reads
// them. Strides over one token or one head do not count.
int check_in_q(const Heads& q, const Heads& out, long long tokens) {
  if (q.p == out.p && ((tokens > 1 && q.ts != out.ts) || (q.n > 1 && q.hs != out.hs)))
    return fail(EMB_E_INVAL, "out is q with other strides");
  return EMB_OK;
}

int check_workspace(const void* ws, size_t ws_bytes, size_t need) {
  if (!ws) return fail(EMB_E_INVAL, "ws is NULL");
  if (!aligned(ws, 16)) return fail(EMB_E_INVAL, "ws is not 16-byte aligned");
  if (ws_bytes < need) return fail(EMB_E_WORKSPACE, "workspace of %zu bytes, need %zu", ws_bytes, need);
  return EMB_OK;
}

int check_step(const emb_history* history, const emb_kv* kv, int32_t seqs, int32_t width) {
  if (!history) return fail(EMB_E_INVAL, "history is NULL");
  if (!kv) return fail(EMB_E_INVAL, "kv is NULL");
  const HistoryView& h = history->v;
  const KvView& c = kv->v;
  if (c.dtype != h.dtype) return fail(EMB_E_DTYPE, "dtype %d, but the cache's is %d", h.dtype, c.dtype);
  if (c.heads != h.kv_heads || c.dim != h.dim)
    return fail(EMB_E_INVAL, "heads of %d x %d, but the cache's are %d x %d", h.kv_heads, h.dim, c.heads, c.dim);
  if (h.q_heads > 32 * h.kv_heads) return fail(EMB_E_INVAL, "more than 32 query heads for a cache head");
  for (long long s : {c.kps, c.kss, c.khs, c.vps, c.vss, c.vhs})
    if (s % 8 != 0) return fail(EMB_E_INVAL, "a stride of the cache is not a multiple of 16 bytes");
  if (!aligned(c.k, 16) || !aligned(c.v, 16)) return fail(EMB_E_INVAL, "the cache is not 16-byte aligned");
  if (seqs < 0 || seqs >= (1 << 24)) return fail(EMB_E_INVAL, "seqs %d not in [0, 2^24)", seqs);
  if (width < 0 || (long long)width * c.page >= (1ll << 30)) return fail(EMB_E_INVAL, "a page table row holds 2^30 slots or more");
  if ((long long)seqs * h.kv_heads >= kMaxBlocks / 2 || (long long)seqs * h.q_heads >= (1ll << 28))
    return fail(EMB_E_INVAL, "too many sequences for one call");
  return EMB_OK;
}

size_t step_lse_offset(const HistoryView& h, int parts, int seqs) {
  return ((size_t)parts * seqs * h.q_heads * h.dim * 4 + 255) & ~size_t(255);
}

}  // namespace

extern "C" {

int emb_layer_norm(int64_t rows, int32_t dim, const void* x, int32_t x_dtype, int64_t x_stride, void* y,
                   int32_t y_dtype, int64_t y_stride, const float* w, const float* b, float eps, void* hip_stream) {
  int rc = check_rows_sizes(rows, dim, EMB_MAX_ROW_DIM);
  if (rc) return rc;
  if ((rc = check_types(x_dtype, y_dtype)) || (rc = check_norm("w", w, eps)) || (rc = check_norm("b", b, eps))) return rc;
  if (rows == 0) return ok();
  const LayerNormArgs a{rows, dim, {x, x_stride, x_dtype}, {y, y_stride, y_dtype}, w, b, eps};
  if ((rc = check_rows("x", a.x)) || (rc = check_rows_out("y", a.y, rows, dim)) || (rc = check_same("x", a.x, "y", a.y)))
    return rc;
  hipError_t e = launch_layer_norm(a, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "layer norm");
  return ok();
}

size_t emb_layer_norm_workspace_bytes(int64_t rows, int32_t dim) {
  if (check_rows_sizes(rows, dim, EMB_MAX_ROW_DIM)) return 0;
  return (size_t)layer_norm_back_blocks(rows) * 2 * dim * sizeof(float);
}

int emb_layer_norm_backward(int64_t rows, int32_t dim, const void* x, int32_t x_dtype, int64_t x_stride,
                            const void* dy, int32_t y_dtype, int64_t dy_stride, void* dx, int64_t dx_stride,
                            const float* w, float eps, void* ws, size_t ws_bytes, float* dw, float* db,
                            void* hip_stream) {
  int rc = check_rows_sizes(rows, dim, EMB_MAX_ROW_DIM);
  if (rc) return rc;
  if ((rc = check_types(x_dtype, y_dtype)) || (rc = check_norm("w", w, eps))) return rc;
  if (!aligned(dw, 4) || !aligned(db, 4)) return fail(EMB_E_INVAL, "dw/db are misaligned");
  const LayerNormBackArgs a{rows, dim, {x, x_stride, x_dtype}, {dy, dy_stride, y_dtype}, {dx, dx_stride, x_dtype},
                            w, eps, static_cast<float*>(ws), dw, db};
  if (rows > 0) {
    if ((rc = check_rows("x", a.x)) || (rc = check_rows("dy", a.dy)) || (rc = check_rows_out("dx", a.dx, rows, dim)) ||
        (rc = check_same("x", a.x, "dx", a.dx)) || (rc = check_same("dy", a.dy, "dx", a.dx)))
      return rc;
    const size_t need = emb_layer_norm_workspace_bytes(rows, dim);
    if (!ws) return fail(EMB_E_INVAL, "ws is NULL");
    if (!aligned(ws, 16)) return fail(EMB_E_INVAL, "ws is not 16-byte aligned");
    if (ws_bytes < need) return fail(EMB_E_WORKSPACE, "workspace of %zu bytes, need %zu", ws_bytes, need);
  }
  hipError_t e = launch_layer_norm_back(a, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "gradient of layer norm");
  return ok();
}

int emb_dropout(int64_t rows, int32_t dim, int32_t dtype, const void* x, int64_t x_stride, const void* residual,
                int64_t residual_stride, void* y, int64_t y_stride, double p, uint64_t seed, const int64_t* step,
                void* hip_stream) {
  int rc = check_rows_sizes(rows, dim, (1ll << 31) - 1);
  if (rc) return rc;
  if ((rc = check_dtype(dtype))) return rc;
  if (!(p >= 0.0 && p <= 1.0)) return fail(EMB_E_INVAL, "p is not in [0, 1]");
  if (!aligned(step, 8)) return fail(EMB_E_INVAL, "step is misaligned");
  if (rows == 0) return ok();
  const uint64_t t = (uint64_t)std::floor(p * 0x1p32 + 0.5);
  const float scale = t >> 32 ? 0.f : (float)(1.0 / (1.0 - (double)t * 0x1p-32));
  const DropoutArgs a{rows, dim, {x, x_stride, dtype}, {residual, residual_stride, dtype}, {y, y_stride, dtype},
                      t, scale, seed, reinterpret_cast<const long long*>(step)};
  if ((rc = check_rows("x", a.x)) || (rc = check_rows_out("y", a.y, rows, dim)) || (rc = check_same("x", a.x, "y", a.y)))
    return rc;
  if (residual && ((rc = check_rows("residual", a.res)) || (rc = check_same("residual", a.res, "y", a.y)))) return rc;
  hipError_t e = launch_dropout(a, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "dropout");
  return ok();
}

int emb_create_history(const emb_history_desc* d, emb_history** out) {
  if (!out) return fail(EMB_E_INVAL, "out is NULL");
  *out = nullptr;
  if (!d) return fail(EMB_E_INVAL, "desc is NULL");
  if (d->dtype != EMB_BF16 && d->dtype != EMB_F16) return fail(EMB_E_DTYPE, "dtype %d is not bf16 or fp16", d->dtype);
  if (d->dim != 64 && d->dim != 96 && d->dim != 128) return fail(EMB_E_INVAL, "dim %d: 64, 96 or 128", d->dim);
  if (d->kv_heads < 1 || d->q_heads < 1 || d->q_heads > 65535 || d->q_heads % d->kv_heads != 0 ||
      d->q_heads / d->kv_heads > 64)
    return fail(EMB_E_INVAL, "q_heads %d is not 1..64 times kv_heads %d, or beyond 65535", d->q_heads, d->kv_heads);
  if (!(d->scale >= 0x1p-100f && d->scale <= 0x1p100f)) return fail(EMB_E_INVAL, "scale is not in [2^-100, 2^100]");
  if (d->buckets < 0 || d->buckets > EMB_MAX_BUCKETS)
    return fail(EMB_E_INVAL, "buckets %d not in [0, %d]", d->buckets, EMB_MAX_BUCKETS);
  if (d->buckets == 0 ? d->exact != 0 : d->exact < 1 || d->exact > d->buckets)
    return fail(EMB_E_INVAL, "exact %d with %d buckets", d->exact, d->buckets);
  if (d->exact < d->buckets && (d->far <= d->exact || d->far > (1 << 30)))
    return fail(EMB_E_INVAL, "far %d not in (exact %d, 2^30]", d->far, d->exact);
  if (d->reserved != 0) return fail(EMB_E_INVAL, "reserved must be 0");
  if (!aligned(d->error, 4)) return fail(EMB_E_INVAL, "error is misaligned");
  emb_history* h = new (std::nothrow) emb_history();
  if (!h) return fail(EMB_E_INVAL, "out of host memory");
  h->v = HistoryView{d->q_heads, d->kv_heads, d->dim, d->dtype, d->causal != 0, d->scale, make_buckets(*d), d->error};
  *out = h;
  return ok();
}

void emb_destroy_history(emb_history* history) { delete history; }

int emb_check_history_error(emb_history* history, void* hip_stream) {
  if (!history) return fail(EMB_E_INVAL, "history is NULL");
  if (!history->v.error) return ok();
  hipError_t e = hipStreamSynchronize(static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
  int flag = 0;
  e = hipMemcpy(&flag, history->v.error, sizeof(int), hipMemcpyDeviceToHost);
  if (e != hipSuccess) return hip_fail(e, "hipMemcpy(history error flag)");
  if (!flag) return ok();
  const int zero = 0;
  e = hipMemcpy(history->v.error, &zero, sizeof(int), hipMemcpyHostToDevice);
  if (e != hipSuccess) return hip_fail(e, "hipMemcpy(clear history error flag)");
  return fail(EMB_E_INVAL, "offsets break their contract (first 0, non-decreasing, last the number of tokens)");
}

int emb_history_attention(emb_history* history, int64_t tokens, const void* q, int64_t q_token_stride,
                          int64_t q_head_stride, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                          const void* v, int64_t v_token_stride, int64_t v_head_stride, void* out,
                          int64_t out_token_stride, int64_t out_head_stride, const int32_t* offsets, int32_t seqs,
                          const float* bias, float* lse, void* hip_stream) {
  int rc = check_ragged(history, tokens, offsets, seqs, bias);
  if (rc) return rc;
  if (!aligned(lse, 4)) return fail(EMB_E_INVAL, "lse is misaligned");
  if (tokens == 0) return ok();
  const HistoryView& h = history->v;
  const HistoryArgs a{h, (int)tokens, seqs, {q, q_token_stride, q_head_stride, h.q_heads},
                      {k, k_token_stride, k_head_stride, h.kv_heads}, {v, v_token_stride, v_head_stride, h.kv_heads},
                      {out, out_token_stride, out_head_stride, h.q_heads}, offsets, bias, lse};
  if ((rc = check_wide("q", a.q, tokens, h, false)) || (rc = check_wide("k", a.k, tokens, h, false)) ||
      (rc = check_wide("v", a.v, tokens, h, false)) || (rc = check_wide("out", a.out, tokens, h, true)) ||
      (rc = check_apart("out", a.out, {a.k, a.v})) || (rc = check_in_q(a.q, a.out, tokens)))
    return rc;
  hipError_t e = launch_history(a, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "attention of histories");
  return ok();
}

size_t emb_history_attention_workspace_bytes(const emb_history* history, int64_t tokens, int32_t seqs) {
  if (!history || tokens < 0 || tokens >= (1ll << 24) || seqs < 0 || seqs >= (1 << 24)) return 0;
  if (too_many(history->v, tokens, seqs)) return 0;
  return history_back_plan(history->v, tokens, seqs).bytes;
}

int emb_history_attention_backward(emb_history* history, int64_t tokens, const void* q, int64_t q_token_stride,
                                   int64_t q_head_stride, const void* k, int64_t k_token_stride,
                                   int64_t k_head_stride, const void* v, int64_t v_token_stride,
                                   int64_t v_head_stride, const void* out, int64_t out_token_stride,
                                   int64_t out_head_stride, const float* lse, const void* dout,
                                   int64_t dout_token_stride, int64_t dout_head_stride, void* dq,
                                   int64_t dq_token_stride, int64_t dq_head_stride, void* dk,
                                   int64_t dk_token_stride, int64_t dk_head_stride, void* dv,
                                   int64_t dv_token_stride, int64_t dv_head_stride, const int32_t* offsets,
                                   int32_t seqs, const float* bias, void* ws, size_t ws_bytes, float* dbias,
                                   void* hip_stream) {
  int rc = check_ragged(history, tokens, offsets, seqs, bias);
  if (rc) return rc;
  const HistoryView& h = history->v;
  if (dbias && (h.buckets.n == 0 || !aligned(dbias, 4))) return fail(EMB_E_INVAL, "dbias without buckets or misaligned");
  if (tokens == 0 && !dbias) return ok();
  HistoryBackArgs a{{h, (int)tokens, seqs, {q, q_token_stride, q_head_stride, h.q_heads},
                     {k, k_token_stride, k_head_stride, h.kv_heads}, {v, v_token_stride, v_head_stride, h.kv_heads},
                     {out, out_token_stride, out_head_stride, h.q_heads}, offsets, bias, const_cast<float*>(lse)},
                    {dout, dout_token_stride, dout_head_stride, h.q_heads},
                    {dq, dq_token_stride, dq_head_stride, h.q_heads}, {dk, dk_token_stride, dk_head_stride, h.kv_heads},
                    {dv, dv_token_stride, dv_head_stride, h.kv_heads}, dbias, nullptr, nullptr};
  if (tokens > 0) {
    if ((rc = check_wide("q", a.f.q, tokens, h, false)) || (rc = check_wide("k", a.f.k, tokens, h, false)) ||
        (rc = check_wide("v", a.f.v, tokens, h, false)) || (rc = check_wide("out", a.f.out, tokens, h, false)) ||
        (rc = check_wide("dout", a.dout, tokens, h, false)) || (rc = check_wide("dq", a.dq, tokens, h, true)) ||
        (rc = check_wide("dk", a.dk, tokens, h, true)) || (rc = check_wide("dv", a.dv, tokens, h, true)))
      return rc;
    if (!lse || !aligned(lse, 4)) return fail(EMB_E_INVAL, "lse is NULL or misaligned");
    const HistoryBackPlan p = history_back_plan(h, tokens, seqs);
    if ((rc = check_workspace(ws, ws_bytes, p.bytes))) return rc;
    if ((rc = check_apart("dq", a.dq, {a.f.q, a.f.k, a.f.v, a.f.out, a.dout, a.dk, a.dv})) ||
        (rc = check_apart("dk", a.dk, {a.f.q, a.f.k, a.f.v, a.f.out, a.dout, a.dv})) ||
        (rc = check_apart("dv", a.dv, {a.f.q, a.f.k, a.f.v, a.f.out, a.dout})))
      return rc;
    a.rows = static_cast<float*>(ws);
    a.part = reinterpret_cast<float*>(static_cast<char*>(ws) + p.part_off);
  }
  hipError_t e = launch_history_back(a, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "gradient of the attention of histories");
  return ok();
}

size_t emb_history_step_workspace_bytes(const emb_history* history, const emb_kv* kv, int32_t seqs,
                                        int32_t table_width) {
  if (check_step(history, kv, seqs, table_width)) return 0;
  const HistoryView& h = history->v;
  const int parts = history_step_parts(h, kv->v, seqs, table_width);
  if (parts == 1 || seqs == 0) return 16;  // none is read; never 0, which stands for invalid arguments
  return step_lse_offset(h, parts, seqs) + (size_t)parts * seqs * h.q_heads * 4;
}

int emb_history_step(emb_history* history, emb_kv* kv, int32_t seqs, const void* q, int64_t q_token_stride,
                     int64_t q_head_stride, void* out, int64_t out_token_stride, int64_t out_head_stride,
                     const int32_t* lens, const int32_t* table, int32_t table_width, const float* bias, void* ws,
                     size_t ws_bytes, float* lse, void* hip_stream) {
  int rc = check_step(history, kv, seqs, table_width);
  if (rc) return rc;
  const HistoryView& h = history->v;
  if (h.buckets.n > 0 && (!bias || !aligned(bias, 4))) return fail(EMB_E_INVAL, "bias is NULL or misaligned");
  if (h.buckets.n == 0 && bias) return fail(EMB_E_INVAL, "bias without buckets");
  if (!aligned(lse, 4)) return fail(EMB_E_INVAL, "lse is misaligned");
  if (seqs == 0) return ok();
  if (!lens || !aligned(lens, 4)) return fail(EMB_E_INVAL, "lens is NULL or misaligned");
  if (table_width > 0 && (!table || !aligned(table, 4))) return fail(EMB_E_INVAL, "table is NULL or misaligned");
  const int parts = history_step_parts(h, kv->v, seqs, table_width);
  HistoryStepArgs a{h, kv->v, seqs, {q, q_token_stride, q_head_stride, h.q_heads},
                    {out, out_token_stride, out_head_stride, h.q_heads}, lens, table, table_width, bias, lse, parts,
                    static_cast<float*>(ws), nullptr};
  if ((rc = check_wide("q", a.q, seqs, h, false)) || (rc = check_wide("out", a.out, seqs, h, true)) ||
      (rc = check_in_q(a.q, a.out, seqs)))
    return rc;
  if ((rc = check_workspace(ws, ws_bytes, emb_history_step_workspace_bytes(history, kv, seqs, table_width)))) return rc;
  a.part_lse = reinterpret_cast<float*>(static_cast<char*>(ws) + step_lse_offset(h, parts, seqs));
  hipError_t e = launch_history_step(a, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "attention of new items");
  return ok();
}

}  // extern "C"
