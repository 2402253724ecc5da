// C-ABI host layer of the sequence operators (rotary positions, head norms,
// paged cache, attention over a shared prefix): argument validation, the
// rotation's frequencies, workspace sizes and the split of the keys. No C++
// exception crosses the ABI.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "emb.h"
#include "seq_internal.h"

using namespace emb;

struct emb_rotary {
  RotTable t;
};

namespace emb {

int check_dtype(int dtype) {
  if (dtype != EMB_F32 && dtype != EMB_BF16 && dtype != EMB_F16) return fail(EMB_E_DTYPE, "unknown dtype %d", dtype);
  return EMB_OK;
}

// A heads operand: pointer given and on an element boundary, strides that
// reach no other head's or token's elements backwards.
int check_heads(const char* name, const Heads& h, int dtype) {
  if (!h.p) return fail(EMB_E_INVAL, "%s is NULL", name);
  if (!aligned(h.p, esize(dtype))) return fail(EMB_E_INVAL, "%s is not aligned to its elements", name);
  if (h.ts < 0 || h.hs < 0) return fail(EMB_E_INVAL, "%s has a negative stride", name);
  return EMB_OK;
}

// An operand that is written: no two of its heads may share elements.
int check_out(const char* name, const Heads& h, long long tokens, int dim, int dtype) {
  if (int rc = check_heads(name, h, dtype)) return rc;
  typedef __int128 Wide;  // strides may be anything up to 2^63
  const bool heads_apart = h.n <= 1 || h.hs >= dim;
  const bool tokens_apart = tokens <= 1 || h.ts >= (Wide)(h.n - 1) * h.hs + dim;
  // tokens inside heads: [heads][tokens][dim] in memory
  const bool swapped = (tokens <= 1 || h.ts >= dim) && (h.n <= 1 || h.hs >= (Wide)(tokens - 1) * h.ts + dim);
  if (!((heads_apart && tokens_apart) || swapped))
    return fail(EMB_E_INVAL, "%s: heads of strides %lld, %lld overlap", name, h.ts, h.hs);
  return EMB_OK;
}

int check_norm(const char* name, const float* w, float eps) {
  if (w && !aligned(w, 16)) return fail(EMB_E_INVAL, "%s is not 16-byte aligned", name);
  if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(EMB_E_INVAL, "eps must be finite and >= 0");
  return EMB_OK;
}

}  // namespace emb

namespace {

int check_itype(int itype) {
  if (itype != EMB_I32 && itype != EMB_I64) return fail(EMB_E_DTYPE, "itype %d is not EMB_I32/EMB_I64", itype);
  return EMB_OK;
}

// Overlap of two operands is only allowed as the very same view.
int check_in_place(const char* in_name, const Heads& in, const char* out_name, const Heads& out) {
  if (in.p == out.p && (in.ts != out.ts || in.hs != out.hs))
    return fail(EMB_E_INVAL, "%s is %s with other strides", out_name, in_name);
  return EMB_OK;
}

int check_common(const emb_rotary* rot, const void* positions, int itype, int64_t tokens, int dtype, int dim, int hq,
                 int hk) {
  if (!rot) return fail(EMB_E_INVAL, "rot is NULL");
  if (int rc = check_itype(itype)) return rc;
  if (int rc = check_dtype(dtype)) return rc;
  if (tokens < 0 || tokens >= (1ll << 31)) return fail(EMB_E_INVAL, "tokens %lld not in [0, 2^31)", (long long)tokens);
  if (dim < rot->t.rot || dim > EMB_MAX_HEAD_DIM)
    return fail(EMB_E_INVAL, "dim %d not in [rot %d, %d]", dim, rot->t.rot, EMB_MAX_HEAD_DIM);
  if (hq < 0 || hk < 0 || hq > 65535 || hk > 65535)
    return fail(EMB_E_INVAL, "q_heads %d / k_heads %d not in [0, 65535]", hq, hk);
  if (tokens > 0 && hq + hk > 0) {
    if (!positions) return fail(EMB_E_INVAL, "positions is NULL");
    if (!aligned(positions, itype == EMB_I64 ? 8 : 4)) return fail(EMB_E_INVAL, "positions are misaligned");
  }
  return EMB_OK;
}

}  // namespace

namespace emb {

FastDiv fast_div(uint32_t d) {
  uint32_t s = 0;
  while ((1ull << s) < d) ++s;
  return FastDiv{(uint32_t)((1ull << (31 + s)) / d + 1), 31 + s, d};
}

// Blocks of the gradient kernel. Its groups of lanes take 4 heads each; a
// block count that is a multiple of the head groups keeps every group on one
// of them, so that it sums one weight's gradient only. Four blocks per CU hide
// the memory's latency; fewer where there is less work than that.
int norm_rotary_back_blocks(long long tokens, int hq, int hk, int dim) {
  const long long heads = (hq + 3) / 4 + (hk + 3) / 4;
  if (heads == 0 || tokens == 0) return 0;
  const long long work = (tokens * heads + 7) / 8;
  const long long n = std::min<long long>(work, 1024);
  return (int)((n + heads - 1) / heads * heads);
}

// Parts of the keys. A launch should give every CU several blocks, so few
// query rows mean many parts; but each part writes and reads back an fp32
// partial output, so a part is never below 256 slots of a prefix or 128 of an
// own sequence (8 queries over 4096 slots: 512 or 128 slots a part measure the
// same, over 1000 slots 512 take 20 us for 17).
//
// Short own sequences are taken by the blocks of their rows' prefix, spread over
// its parts: with one part the result is written directly, without partial
// outputs (24 users' 1200 candidates: 142 -> 125 us). Beyond kOwnInPrefix slots
// of table width they would hold these blocks up, and get blocks of their own.
constexpr long long kOwnInPrefix = 256;

PrefixPlan prefix_plan(const KvView& kv, long long tokens, int q_heads, int groups, int pwidth,
                       int width) {
  PrefixPlan p{};
  if (tokens == 0) return p;
  const int m = q_heads / kv.heads;
  const long long pcap = groups > 0 ? (long long)pwidth * kv.page : 0;
  const long long ocap = (long long)width * kv.page;
  const bool with_own = pcap > 0 && ocap <= kOwnInPrefix;
  if (pcap > 0) {
    // Rows of one group and cache head, on average. The wide tiles fetch 4 or 8
    // slots of a page at a time, with 32-bit offsets (in 16 bytes) inside a page.
    const long long slots = std::max(kv.kss, kv.vss), step = std::max(kv.kps, kv.vps);
    p.wide = tokens * m > 64ll * groups && kv.page % 8 == 0 && slots * kv.page < (1ll << 31) && step < (1ll << 35);
    const int rows = p.wide ? 128 : 32;
    const long long tiles = std::max<long long>(groups, (tokens * m + rows - 1) / rows);
    const long long want = (512 + tiles * kv.heads - 1) / (tiles * kv.heads);
    // an own tile of 32 slots takes a wave about the time of 64 prefix slots
    const long long own = with_own ? std::max(1, 32 / m) * ((ocap + 31) / 32) * 64 : 0;
    p.nps = (int)std::max<long long>(1, std::min<long long>({want, (pcap + own + 255) / 256, 32}));
    p.prefix_tiles = groups + tokens * m / rows;
    p.prefix_blocks = p.prefix_tiles * kv.heads * p.nps;
    if (p.wide) p.prefix_blocks = (p.prefix_blocks + 7) / 8 * 8;
  }
  if (!with_own) {
    p.own_tiles = (tokens * m + 31) / 32;
    const long long waves = p.own_tiles * kv.heads;
    const long long want = (2048 + waves - 1) / waves;
    p.nos = (int)std::max<long long>(1, std::min<long long>({want, (ocap + 127) / 128, 32}));
    p.own_blocks = (waves * p.nos + 3) / 4;
  }
  // the size does not tell whether the prefix blocks take the own slots along
  const size_t rows = (size_t)tokens * q_heads * (p.nps + std::max(p.nos, 1));
  p.lse_off = (rows * kv.dim * 4 + 255) & ~size_t(255);
  p.bytes = p.lse_off + ((rows * 4 + 255) & ~size_t(255));
  return p;
}

}  // namespace emb

extern "C" {

int emb_create_rotary(const emb_rotary_desc* d, emb_rotary** out) {
  if (!out) return fail(EMB_E_INVAL, "out is NULL");
  *out = nullptr;
  if (!d) return fail(EMB_E_INVAL, "desc is NULL");
  if (d->rot < 2 || d->rot > EMB_MAX_ROT || d->rot % 2 != 0)
    return fail(EMB_E_INVAL, "rot %d is not an even number in [2, %d]", d->rot, EMB_MAX_ROT);
  if (d->layout != EMB_ROT_HALF && d->layout != EMB_ROT_INTERLEAVED)
    return fail(EMB_E_INVAL, "unknown layout %d", d->layout);
  if (d->scaling < EMB_ROT_NONE || d->scaling > EMB_ROT_BANDS)
    return fail(EMB_E_INVAL, "unknown scaling %d", d->scaling);
  if (d->reserved != 0) return fail(EMB_E_INVAL, "reserved must be 0");
  if (!(d->base > 1.0) || !std::isfinite(d->base)) return fail(EMB_E_INVAL, "base must be finite and > 1");
  if (!std::isfinite(d->magnitude) || d->magnitude == 0.0)
    return fail(EMB_E_INVAL, "magnitude must be finite and not 0");
  if (d->scaling != EMB_ROT_NONE && (!(d->factor > 0.0) || !std::isfinite(d->factor)))
    return fail(EMB_E_INVAL, "factor must be finite and > 0");
  if (d->scaling == EMB_ROT_BASE && d->rot < 4) return fail(EMB_E_INVAL, "base scaling needs rot >= 4");
  const bool bands = d->scaling == EMB_ROT_PARTS || d->scaling == EMB_ROT_BANDS;
  if (bands && (!(d->original_len > 0.0) || !std::isfinite(d->original_len)))
    return fail(EMB_E_INVAL, "original_len must be finite and > 0");
  if (bands && (!(d->turns_low > 0.0) || !(d->turns_high > d->turns_low) || !std::isfinite(d->turns_high)))
    return fail(EMB_E_INVAL, "need 0 < turns_low < turns_high");
  emb_rotary* r = new (std::nothrow) emb_rotary();
  if (!r) return fail(EMB_E_INVAL, "out of host memory");
  const long double two_pi = 6.283185307179586476925286766559005768L;
  long double base = d->base;
  if (d->scaling == EMB_ROT_BASE) base *= powl(d->factor, (long double)d->rot / (d->rot - 2));
  for (int i = 0; i < d->rot / 2; ++i) {
    long double f = powl(base, -2.0L * i / d->rot);
    if (d->scaling == EMB_ROT_LINEAR) f /= d->factor;
    if (bands) {
      const long double turns = d->original_len * f / two_pi;
      const long double lo = d->turns_low, hi = d->turns_high;
      long double keep = d->scaling == EMB_ROT_PARTS ? logl(turns / lo) / logl(hi / lo) : (turns - lo) / (hi - lo);
      keep = std::min(1.0L, std::max(0.0L, keep));
      f = f * keep + f / d->factor * (1.0L - keep);
    }
    long double frac = f / two_pi;
    frac -= floorl(frac);  // whole turns per position change nothing
    const long double scaled = roundl(frac * 0x1p64L);
    r->t.turn[i] = scaled >= 0x1p64L ? 0 : (uint64_t)scaled;
  }
  r->t.mag = (float)d->magnitude;
  r->t.rot = d->rot;
  r->t.layout = d->layout;
  *out = r;
  return ok();
}

void emb_destroy_rotary(emb_rotary* rot) { delete rot; }

static int norm_rotary(const emb_rotary* rot, NormRotaryArgs& a, void* hip_stream) {
  int rc = check_common(rot, a.positions, a.itype, a.tokens, a.dtype, a.dim, a.q.n, a.k.n);
  if (rc) return rc;
  if (a.norm && ((rc = check_norm("wq", a.wq, a.eps)) || (rc = check_norm("wk", a.wk, a.eps)))) return rc;
  if (a.tokens == 0 || a.q.n + a.k.n == 0) return ok();
  if (a.q.n > 0 && ((rc = check_heads("q", a.q, a.dtype)) || (rc = check_out("q_out", a.qo, a.tokens, a.dim, a.dtype)) ||
                    (rc = check_in_place("q", a.q, "q_out", a.qo))))
    return rc;
  if (a.k.n > 0 && ((rc = check_heads("k", a.k, a.dtype)) || (rc = check_out("k_out", a.ko, a.tokens, a.dim, a.dtype)) ||
                    (rc = check_in_place("k", a.k, "k_out", a.ko))))
    return rc;
  hipError_t e = launch_norm_rotary(a, rot->t, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, a.norm ? "head norm and rotation" : "rotation");
  return ok();
}

int emb_rotary_apply(const emb_rotary* rot, const void* positions, int32_t itype, int64_t tokens, int32_t dtype,
                     int32_t dim, const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                     int64_t q_out_token_stride, int64_t q_out_head_stride, int32_t q_heads, const void* k,
                     int64_t k_token_stride, int64_t k_head_stride, void* k_out, int64_t k_out_token_stride,
                     int64_t k_out_head_stride, int32_t k_heads, int32_t inverse, void* hip_stream) {
  NormRotaryArgs a{positions, itype, tokens, dtype, dim,
                   {q, q_token_stride, q_head_stride, q_heads},
                   {q_out, q_out_token_stride, q_out_head_stride, q_heads},
                   {k, k_token_stride, k_head_stride, k_heads},
                   {k_out, k_out_token_stride, k_out_head_stride, k_heads},
                   inverse != 0, 0, nullptr, nullptr, 0.f};
  return norm_rotary(rot, a, hip_stream);
}

int emb_qk_norm_rotary(const emb_rotary* rot, const void* positions, int32_t itype, int64_t tokens, int32_t dtype,
                       int32_t dim, const void* q, int64_t q_token_stride, int64_t q_head_stride, void* q_out,
                       int64_t q_out_token_stride, int64_t q_out_head_stride, int32_t q_heads, const void* k,
                       int64_t k_token_stride, int64_t k_head_stride, void* k_out, int64_t k_out_token_stride,
                       int64_t k_out_head_stride, int32_t k_heads, const float* wq, const float* wk, float eps,
                       void* hip_stream) {
  NormRotaryArgs a{positions, itype, tokens, dtype, dim,
                   {q, q_token_stride, q_head_stride, q_heads},
                   {q_out, q_out_token_stride, q_out_head_stride, q_heads},
                   {k, k_token_stride, k_head_stride, k_heads},
                   {k_out, k_out_token_stride, k_out_head_stride, k_heads},
                   0, 1, wq, wk, eps};
  return norm_rotary(rot, a, hip_stream);
}

size_t emb_qk_norm_rotary_workspace_bytes(int64_t tokens, int32_t q_heads, int32_t k_heads, int32_t dim) {
  if (tokens < 0 || tokens >= (1ll << 31) || q_heads < 0 || k_heads < 0 || q_heads > 65535 || k_heads > 65535 ||
      dim < 1 || dim > EMB_MAX_HEAD_DIM)
    return 0;
  return (size_t)norm_rotary_back_blocks(tokens, q_heads, k_heads, dim) * 2 * dim * sizeof(float);
}

int emb_qk_norm_rotary_backward(const emb_rotary* rot, const void* positions, int32_t itype, int64_t tokens,
                                int32_t dtype, int32_t dim, const void* q, int64_t q_token_stride,
                                int64_t q_head_stride, const void* dyq, int64_t dyq_token_stride,
                                int64_t dyq_head_stride, void* dq, int64_t dq_token_stride, int64_t dq_head_stride,
                                int32_t q_heads, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                                const void* dyk, int64_t dyk_token_stride, int64_t dyk_head_stride, void* dk,
                                int64_t dk_token_stride, int64_t dk_head_stride, int32_t k_heads, const float* wq,
                                const float* wk, float eps, void* ws, size_t ws_bytes, float* dwq, float* dwk,
                                void* hip_stream) {
  NormRotaryBackArgs a{positions, itype, tokens, dtype, dim,
                       {q, q_token_stride, q_head_stride, q_heads},
                       {dyq, dyq_token_stride, dyq_head_stride, q_heads},
                       {dq, dq_token_stride, dq_head_stride, q_heads},
                       {k, k_token_stride, k_head_stride, k_heads},
                       {dyk, dyk_token_stride, dyk_head_stride, k_heads},
                       {dk, dk_token_stride, dk_head_stride, k_heads},
                       wq, wk, eps, static_cast<float*>(ws), dwq, dwk};
  int rc = check_common(rot, positions, itype, tokens, dtype, dim, q_heads, k_heads);
  if (rc) return rc;
  if ((rc = check_norm("wq", wq, eps)) || (rc = check_norm("wk", wk, eps))) return rc;
  if (!aligned(dwq, 4) || !aligned(dwk, 4)) return fail(EMB_E_INVAL, "dwq/dwk are misaligned");
  const bool any = tokens > 0;
  if (any && q_heads > 0 &&
      ((rc = check_heads("q", a.q, dtype)) || (rc = check_heads("dyq", a.dyq, dtype)) ||
       (rc = check_out("dq", a.dq, tokens, dim, dtype)) || (rc = check_in_place("dyq", a.dyq, "dq", a.dq)) ||
       (rc = check_in_place("q", a.q, "dq", a.dq))))
    return rc;
  if (any && k_heads > 0 &&
      ((rc = check_heads("k", a.k, dtype)) || (rc = check_heads("dyk", a.dyk, dtype)) ||
       (rc = check_out("dk", a.dk, tokens, dim, dtype)) || (rc = check_in_place("dyk", a.dyk, "dk", a.dk)) ||
       (rc = check_in_place("k", a.k, "dk", a.dk))))
    return rc;
  const size_t need = emb_qk_norm_rotary_workspace_bytes(tokens, q_heads, k_heads, dim);
  if (need > 0) {
    if (!ws) return fail(EMB_E_INVAL, "ws is NULL");
    if (!aligned(ws, 16)) return fail(EMB_E_INVAL, "ws is not 16-byte aligned");
    if (ws_bytes < need) return fail(EMB_E_WORKSPACE, "workspace of %zu bytes, need %zu", ws_bytes, need);
  } else if (!dwq && !dwk) {
    return ok();
  }
  hipError_t e = launch_norm_rotary_back(a, rot->t, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "gradient of head norm and rotation");
  return ok();
}

int emb_create_kv(const emb_kv_desc* d, emb_kv** out) {
  if (!out) return fail(EMB_E_INVAL, "out is NULL");
  *out = nullptr;
  if (!d) return fail(EMB_E_INVAL, "desc is NULL");
  if (int rc = check_dtype(d->dtype)) return rc;
  if (!d->k || !d->v) return fail(EMB_E_INVAL, "k or v is NULL");
  if (!aligned(d->k, esize(d->dtype)) || !aligned(d->v, esize(d->dtype)))
    return fail(EMB_E_INVAL, "k or v is not aligned to its elements");
  if (d->pages < 1 || d->pages >= (1ll << 31)) return fail(EMB_E_INVAL, "pages %lld not in [1, 2^31)", (long long)d->pages);
  if (d->page < 1 || d->page > (1 << 20)) return fail(EMB_E_INVAL, "page %d not in [1, 2^20]", d->page);
  if (d->heads < 1 || d->heads > 65535) return fail(EMB_E_INVAL, "heads %d not in [1, 65535]", d->heads);
  if (d->dim < 1 || d->dim > EMB_MAX_HEAD_DIM) return fail(EMB_E_INVAL, "dim %d not in [1, %d]", d->dim, EMB_MAX_HEAD_DIM);
  for (int64_t s : {d->k_page_stride, d->k_slot_stride, d->k_head_stride, d->v_page_stride, d->v_slot_stride,
                    d->v_head_stride})
    if (s < 0) return fail(EMB_E_INVAL, "a stride of the cache is negative");
  if (!aligned(d->error, 4)) return fail(EMB_E_INVAL, "error is misaligned");
  emb_kv* c = new (std::nothrow) emb_kv();
  if (!c) return fail(EMB_E_INVAL, "out of host memory");
  c->v = KvView{static_cast<char*>(d->k), static_cast<char*>(d->v), d->k_page_stride, d->k_slot_stride,
                d->k_head_stride, d->v_page_stride, d->v_slot_stride, d->v_head_stride, (int)d->pages, d->page,
                d->heads, d->dim, d->dtype, fast_div((uint32_t)d->page), d->error};
  *out = c;
  return ok();
}

void emb_destroy_kv(emb_kv* kv) { delete kv; }

int emb_check_kv_error(emb_kv* kv, void* hip_stream) {
  if (!kv) return fail(EMB_E_INVAL, "kv is NULL");
  if (!kv->v.error) return ok();
  hipError_t e = hipStreamSynchronize(static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "hipStreamSynchronize");
  int flag = 0;
  e = hipMemcpy(&flag, kv->v.error, sizeof(int), hipMemcpyDeviceToHost);
  if (e != hipSuccess) return hip_fail(e, "hipMemcpy(cache error flag)");
  if (!flag) return ok();
  const int zero = 0;
  e = hipMemcpy(kv->v.error, &zero, sizeof(int), hipMemcpyHostToDevice);
  if (e != hipSuccess) return hip_fail(e, "hipMemcpy(clear cache error flag)");
  if (flag & kKvBadPage)
    return fail(EMB_E_BOUNDS, "a kernel met a page outside [0, pages) or a length that its page table does not hold");
  return fail(EMB_E_INVAL, "offsets break their contract (first 0, non-decreasing, last the number of tokens or "
                           "sequences)");
}

static int check_cache(const emb_kv* kv, int dtype, int heads, int dim) {
  if (dtype != kv->v.dtype) return fail(EMB_E_DTYPE, "dtype %d, but the cache's is %d", dtype, kv->v.dtype);
  if (heads != kv->v.heads || dim != kv->v.dim)
    return fail(EMB_E_INVAL, "heads of %d x %d, but the cache's are %d x %d", heads, dim, kv->v.heads, kv->v.dim);
  return EMB_OK;
}

static int check_seqs(const int32_t* offsets, int64_t tokens, int32_t seqs, const int32_t* lens, const int32_t* table,
                      int32_t width) {
  if (tokens < 0 || tokens >= (1ll << 31)) return fail(EMB_E_INVAL, "tokens %lld not in [0, 2^31)", (long long)tokens);
  if (seqs < 0) return fail(EMB_E_INVAL, "seqs %d < 0", seqs);
  if (!offsets && seqs != tokens)
    return fail(EMB_E_INVAL, "without offsets each sequence has one token, but seqs %d != tokens %lld", seqs,
                (long long)tokens);
  if (seqs == 0 && tokens > 0) return fail(EMB_E_INVAL, "tokens without a sequence");
  if (width < 0) return fail(EMB_E_INVAL, "table_width %d < 0", width);
  if (tokens == 0) return EMB_OK;
  if (!lens || !aligned(lens, 4)) return fail(EMB_E_INVAL, "lens is NULL or misaligned");
  if (width > 0 && (!table || !aligned(table, 4))) return fail(EMB_E_INVAL, "table is NULL or misaligned");
  if (!aligned(offsets, 4)) return fail(EMB_E_INVAL, "offsets are misaligned");
  return EMB_OK;
}

int emb_kv_append(emb_kv* kv, const emb_rotary* rot, int64_t tokens, int32_t dtype, int32_t heads, int32_t dim,
                  const void* k, int64_t k_token_stride, int64_t k_head_stride, const void* v, int64_t v_token_stride, int64_t v_head_stride,
                  const int32_t* offsets, int32_t seqs, const int32_t* lens, const int32_t* table,
                  int32_t table_width, const void* positions, int32_t itype, int32_t norm, const float* wk,
                  float eps, void* hip_stream) {
  if (!kv) return fail(EMB_E_INVAL, "kv is NULL");
  int rc = check_cache(kv, dtype, heads, dim);
  if (rc) return rc;
  if ((rc = check_seqs(offsets, tokens, seqs, lens, table, table_width))) return rc;
  if ((rc = check_itype(itype))) return rc;
  if (rot && rot->t.rot > kv->v.dim) return fail(EMB_E_INVAL, "rot %d > dim %d", rot->t.rot, kv->v.dim);
  if (!rot && positions) return fail(EMB_E_INVAL, "positions without a rotation");
  if (!aligned(positions, itype == EMB_I64 ? 8 : 4)) return fail(EMB_E_INVAL, "positions are misaligned");
  if (norm && (rc = check_norm("wk", wk, eps))) return rc;
  if (!norm && wk) return fail(EMB_E_INVAL, "wk without norm");
  if (tokens == 0) return ok();
  AppendArgs a{kv->v, tokens, {k, k_token_stride, k_head_stride, kv->v.heads},
               {v, v_token_stride, v_head_stride, kv->v.heads}, offsets, seqs, lens, table, table_width,
               positions, itype, norm != 0, wk, eps};
  if ((rc = check_heads("k", a.k, kv->v.dtype)) || (rc = check_heads("v", a.v, kv->v.dtype))) return rc;
  static const RotTable none{};
  hipError_t e = launch_kv_append(a, rot ? rot->t : none, static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "append to the cache");
  return ok();
}

static int check_prefix_sizes(const emb_kv* kv, int64_t tokens, int32_t q_heads, int32_t groups, int32_t pwidth,
                              int32_t width) {
  if (!kv) return fail(EMB_E_INVAL, "kv is NULL");
  const KvView& c = kv->v;
  if (c.dtype == EMB_F32) return fail(EMB_E_DTYPE, "attention needs a bf16 or fp16 cache");
  if (c.dim != 64 && c.dim != 96 && c.dim != 128) return fail(EMB_E_INVAL, "attention over dim %d: 64, 96 or 128", c.dim);
  for (long long s : {c.kps, c.kss, c.khs, c.vps, c.vss, c.vhs})
    if (s % 8 != 0) return fail(EMB_E_INVAL, "a stride of the cache is not a multiple of 16 bytes");
  if (!aligned(c.k, 16) || !aligned(c.v, 16)) return fail(EMB_E_INVAL, "the cache is not 16-byte aligned");
  if (tokens < 0 || tokens >= (1ll << 24)) return fail(EMB_E_INVAL, "tokens %lld not in [0, 2^24)", (long long)tokens);
  if (q_heads < 1 || q_heads % c.heads != 0 || q_heads / c.heads > 64)
    return fail(EMB_E_INVAL, "q_heads %d is not 1..64 times the cache's heads %d", q_heads, c.heads);
  if (tokens * (long long)q_heads >= (1ll << 31)) return fail(EMB_E_INVAL, "tokens * q_heads must be < 2^31");
  if (groups < 0 || pwidth < 0 || width < 0) return fail(EMB_E_INVAL, "negative groups or table width");
  if ((long long)pwidth * c.page >= (1ll << 30) || (long long)width * c.page >= (1ll << 30))
    return fail(EMB_E_INVAL, "a page table row holds 2^30 slots or more");
  return EMB_OK;
}

size_t emb_prefix_attention_workspace_bytes(const emb_kv* kv, int64_t tokens, int32_t q_heads, int32_t groups,
                                            int32_t prefix_width, int32_t table_width) {
  if (check_prefix_sizes(kv, tokens, q_heads, groups, prefix_width, table_width)) return 0;
  return prefix_plan(kv->v, tokens, q_heads, groups, prefix_width, table_width).bytes;
}

int emb_prefix_attention(emb_kv* kv, int64_t tokens, int32_t dtype, int32_t dim, const void* q,
                         int64_t q_token_stride, int64_t q_head_stride, void* out, int64_t out_token_stride, int64_t out_head_stride, int32_t q_heads, float scale,
                         const int32_t* offsets, int32_t seqs, const int32_t* lens, const int32_t* table,
                         int32_t table_width, const int32_t* group_offsets, int32_t groups,
                         const int32_t* prefix_lens, const int32_t* prefix_table, int32_t prefix_width, void* ws,
                         size_t ws_bytes, float* lse, void* hip_stream) {
  int rc = check_prefix_sizes(kv, tokens, q_heads, groups, prefix_width, table_width);
  if (rc) return rc;
  if ((rc = check_cache(kv, dtype, kv->v.heads, dim))) return rc;
  if ((rc = check_seqs(offsets, tokens, seqs, lens, table, table_width))) return rc;
  // the kernels hold scale * log2(e) in fp32
  if (!(std::fabs(scale) <= 0x1p127f)) return fail(EMB_E_INVAL, "scale is not a number within +- 2^127");
  if (groups > 0) {
    if (!group_offsets || !prefix_lens || !aligned(group_offsets, 4) || !aligned(prefix_lens, 4))
      return fail(EMB_E_INVAL, "group_offsets/prefix_lens is NULL or misaligned");
    if (prefix_width > 0 && (!prefix_table || !aligned(prefix_table, 4)))
      return fail(EMB_E_INVAL, "prefix_table is NULL or misaligned");
  } else if (group_offsets || prefix_lens || prefix_table) {
    return fail(EMB_E_INVAL, "prefix arguments without groups");
  }
  if (tokens == 0) return ok();
  PrefixArgs a{kv->v, (int)tokens, q_heads, {q, q_token_stride, q_head_stride, q_heads},
               {out, out_token_stride, out_head_stride, q_heads}, scale, offsets, seqs, lens, table, table_width,
               group_offsets, groups, prefix_lens, prefix_table, prefix_width, lse};
  if ((rc = check_heads("q", a.q, kv->v.dtype)) || (rc = check_out("out", a.out, tokens, kv->v.dim, kv->v.dtype)))
    return rc;
  for (const Heads* h : {&a.q, &a.out})
    if (!aligned(h->p, 16) || h->ts % 8 != 0 || h->hs % 8 != 0)
      return fail(EMB_E_INVAL, "q and out need 16-byte alignment and strides of multiples of 16 bytes");
  if (!aligned(lse, 4)) return fail(EMB_E_INVAL, "lse is misaligned");
  const PrefixPlan p = prefix_plan(kv->v, tokens, q_heads, groups, prefix_width, table_width);
  if (p.prefix_blocks + p.own_blocks >= (1ll << 24) || p.own_tiles * kv->v.heads * std::max(p.nos, 1) >= (1ll << 31))
    return fail(EMB_E_INVAL, "too many sequences or groups for one call");
  if (!ws) return fail(EMB_E_INVAL, "ws is NULL");
  if (!aligned(ws, 16)) return fail(EMB_E_INVAL, "ws is not 16-byte aligned");
  if (ws_bytes < p.bytes) return fail(EMB_E_WORKSPACE, "workspace of %zu bytes, need %zu", ws_bytes, p.bytes);
  hipError_t e = launch_prefix_attention(a, p, static_cast<char*>(ws), static_cast<hipStream_t>(hip_stream));
  if (e != hipSuccess) return hip_fail(e, "prefix attention");
  return ok();
}

}  // extern "C"
