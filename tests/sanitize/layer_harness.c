/* Drives the host side of the history layer (emb_layer.cpp) without a device:
 * descriptors over their whole range, refusals, and accepted calls as far as
 * the launch, which is a stub that counts. Built with the host sanitizers by
 * tests/test_layer_sanitizers.py. Prints "layer harness ok: N checks" and exits
 * 0, or reports the first mismatch and exits 1. */
#include <float.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "emb.h"

int stub_launches(void);
int stub_bucket_start(int i);

static int g_checks = 0;

#define CHECK(cond)                                                                                   \
  do {                                                                                                \
    ++g_checks;                                                                                       \
    if (!(cond)) {                                                                                    \
      fprintf(stderr, "line %d: check failed: %s (%s)\n", __LINE__, #cond, emb_last_error());         \
      return 1;                                                                                       \
    }                                                                                                 \
  } while (0)
#define EXPECT(call, code)                                            \
  do {                                                                \
    CHECK((call) == (code));                                          \
    CHECK((code) == EMB_OK || emb_last_error()[0] != '\0');           \
  } while (0)

/* 16-byte aligned addresses, never dereferenced */
#define FAKE(k) ((void*)(uintptr_t)(0x100000u + 0x10000u * (unsigned)(k)))

static emb_history_desc desc(int q_heads, int kv_heads, int dim, int causal, int buckets, int exact, int far) {
  emb_history_desc d;
  memset(&d, 0, sizeof d);
  d.q_heads = q_heads;
  d.kv_heads = kv_heads;
  d.dim = dim;
  d.dtype = EMB_BF16;
  d.causal = causal;
  d.buckets = buckets;
  d.exact = exact;
  d.far = far;
  d.scale = 0.125f;
  return d;
}

static int attend(emb_history* h, int64_t tokens, int32_t seqs, const float* bias) {
  return emb_history_attention(h, tokens, FAKE(1), 512, 64, FAKE(2), 128, 64, FAKE(3), 128, 64, FAKE(4), 512, 64, FAKE(5),
                               seqs, bias, FAKE(6), NULL);
}

/* Bounds of the buckets: they increase from 0 on, whole numbers up to `exact`, and end at the largest int; each one
 * holds its formula's value to a part in 10^9. */
static int buckets_of(int buckets, int exact, int far) {
  emb_history_desc d = desc(8, 2, 64, 1, buckets, exact, far);
  emb_history* h = NULL;
  EXPECT(emb_create_history(&d, &h), EMB_OK);
  EXPECT(attend(h, 10, 1, FAKE(7)), EMB_OK);
  for (int i = 0; i < buckets; ++i) {
    int at = stub_bucket_start(i);
    if (i <= exact) {
      CHECK(at == i);
    } else {
      double x = exact * pow((double)far / exact, (double)(i - exact) / (buckets - exact));
      CHECK(at >= stub_bucket_start(i - 1) && at <= far);
      CHECK(at >= x * (1 - 1e-9) && at - 1 < x * (1 + 1e-9));
    }
  }
  CHECK(stub_bucket_start(buckets) == INT32_MAX);
  emb_destroy_history(h);
  return 0;
}

static int descriptors(void) {
  const int n[] = {1, 2, 3, 7, 32, 64, 127, 128};
  for (unsigned i = 0; i < sizeof n / sizeof *n; ++i)
    for (int exact = 1; exact <= n[i]; exact += exact < 4 ? 1 : exact / 2) {
      const int far[] = {exact + 1, exact + 2, 2 * exact + 1, 1000, 1 << 20, (1 << 30) - 1, 1 << 30};
      for (unsigned f = 0; f < sizeof far / sizeof *far; ++f)
        if (far[f] > exact && buckets_of(n[i], exact, far[f])) return 1;
    }
  if (buckets_of(128, 128, 0) || buckets_of(1, 1, -5)) return 1;
  emb_history* h = NULL;
  emb_history_desc bad[] = {desc(8, 2, 64, 1, -1, 1, 9),      desc(8, 2, 64, 1, EMB_MAX_BUCKETS + 1, 1, 9),
                            desc(8, 2, 64, 1, 8, 9, 20),      desc(8, 2, 64, 1, 8, 0, 20),
                            desc(8, 2, 64, 1, 8, 4, 4),       desc(8, 2, 64, 1, 8, 4, INT32_MAX),
                            desc(8, 2, 64, 1, 8, 4, INT32_MIN), desc(INT32_MAX, 1, 64, 1, 0, 0, 0),
                            desc(8, INT32_MIN, 64, 1, 0, 0, 0), desc(INT32_MIN, -1, 64, 1, 0, 0, 0),
                            desc(8, 2, 63, 1, 0, 0, 0),       desc(65536, 65536, 64, 1, 0, 0, 0)};
  for (unsigned i = 0; i < sizeof bad / sizeof *bad; ++i) {
    EXPECT(emb_create_history(&bad[i], &h), EMB_E_INVAL);
    CHECK(h == NULL);
  }
  EXPECT(emb_create_history(NULL, &h), EMB_E_INVAL);
  EXPECT(emb_create_history(&bad[0], NULL), EMB_E_INVAL);
  emb_destroy_history(NULL);
  return 0;
}

static int attention(void) {
  emb_history_desc d = desc(8, 2, 64, 0, 32, 16, 128);
  emb_history *h = NULL, *widest = NULL;
  EXPECT(emb_create_history(&d, &h), EMB_OK);
  d = desc(65535, 65535, 128, 0, 128, 1, 1 << 30);
  EXPECT(emb_create_history(&d, &widest), EMB_OK);
  const int64_t tokens[] = {0, 1, 63, (1 << 24) - 1, 1 << 24, INT64_MAX, INT64_MIN, -1};
  const int32_t seqs[] = {0, 1, 200, (1 << 21) - 2, (1 << 24) - 1, 1 << 24, INT32_MAX, INT32_MIN};
  for (unsigned i = 0; i < 8; ++i)
    for (unsigned j = 0; j < 8; ++j) {
      const int64_t t = tokens[i];
      const int32_t s = seqs[j];
      const int valid = t >= 0 && t < 1 << 24 && s >= 0 && s < 1 << 24 && (s + t / 64) * 8 < 1 << 24 && t * 8 < (1ll << 31);
      const int before = stub_launches();
      EXPECT(attend(h, t, s, FAKE(7)), valid && (s > 0 || t == 0) ? EMB_OK : EMB_E_INVAL);
      CHECK(stub_launches() - before == (valid && s > 0 && t > 0));
      CHECK((emb_history_attention_workspace_bytes(h, t, s) > 0) == valid);
      (void)emb_history_attention_workspace_bytes(widest, t, s);
      (void)attend(widest, t, s, FAKE(7));
    }
  CHECK(emb_history_attention_workspace_bytes(NULL, 1, 1) == 0);
  EXPECT(attend(NULL, 1, 1, FAKE(7)), EMB_E_INVAL);
  EXPECT(attend(h, 1, 1, NULL), EMB_E_INVAL);
  /* strides at their bounds */
  EXPECT(emb_history_attention(h, 2, FAKE(1), (1 << 24) - 8, INT64_MAX - 7, FAKE(2), 128, 64, FAKE(3), 128, 64, FAKE(4), 512,
                               64, FAKE(5), 1, FAKE(7), NULL, NULL), EMB_OK);
  EXPECT(emb_history_attention(h, 2, FAKE(1), INT64_MAX - 7, 64, FAKE(2), 128, 64, FAKE(3), 128, 64, FAKE(4), 512, 64,
                               FAKE(5), 1, FAKE(7), NULL, NULL), EMB_E_INVAL);
  EXPECT(emb_history_attention(h, 2, FAKE(1), 512, 64, FAKE(2), INT64_MIN, 64, FAKE(3), 128, 64, FAKE(4), 512, 64, FAKE(5),
                               1, FAKE(7), NULL, NULL), EMB_E_INVAL);
  (void)emb_history_attention(h, 2, FAKE(1), 512, 64, FAKE(2), 128, 64, FAKE(3), 128, 64, FAKE(4), INT64_MAX - 7, INT64_MAX - 7,
                              FAKE(5), 1, FAKE(7), NULL, NULL);
  for (int64_t t = 0; t <= 2; ++t)
    for (int grad = 0; grad < 2; ++grad) {
      const int before = stub_launches();
      EXPECT(emb_history_attention_backward(h, t, FAKE(1), 512, 64, FAKE(2), 128, 64, FAKE(3), 128, 64, FAKE(4), 512, 64,
                                            FAKE(6), FAKE(8), 512, 64, FAKE(9), 512, 64, FAKE(10), 128, 64, FAKE(11), 128,
                                            64, FAKE(5), 1, FAKE(7), t ? FAKE(12) : NULL, 4096, grad ? FAKE(13) : NULL, NULL),
             EMB_OK);
      CHECK(stub_launches() - before == (t > 0 || grad));
    }
  EXPECT(emb_history_attention_backward(h, 2, FAKE(1), 512, 64, FAKE(2), 128, 64, FAKE(3), 128, 64, FAKE(4), 512, 64, FAKE(6),
                                        FAKE(8), 512, 64, FAKE(9), 512, 64, FAKE(10), 128, 64, FAKE(11), 128, 64, FAKE(5), 1,
                                        FAKE(7), FAKE(12), 10, NULL, NULL), EMB_E_WORKSPACE);
  EXPECT(emb_check_history_error(h, NULL), EMB_OK);
  EXPECT(emb_check_history_error(NULL, NULL), EMB_E_INVAL);
  emb_destroy_history(h);
  emb_destroy_history(widest);
  return 0;
}

static int step(void) {
  emb_history_desc d = desc(8, 2, 64, 1, 32, 16, 128);
  emb_history* h = NULL;
  EXPECT(emb_create_history(&d, &h), EMB_OK);
  emb_kv_desc k;
  memset(&k, 0, sizeof k);
  k.k = FAKE(20);
  k.v = FAKE(21);
  k.k_page_stride = k.v_page_stride = 16 * 2 * 64;
  k.k_slot_stride = k.v_slot_stride = 64;
  k.k_head_stride = k.v_head_stride = 16 * 64;
  k.pages = 100;
  k.page = 16;
  k.heads = 2;
  k.dim = 64;
  k.dtype = EMB_BF16;
  emb_kv* kv = NULL;
  EXPECT(emb_create_kv(&k, &kv), EMB_OK);
  const int32_t seqs[] = {0, 1, 1000, (1 << 22) - 1, 1 << 22, (1 << 24) - 1, INT32_MAX, INT32_MIN};
  const int32_t width[] = {0, 1, 200, (1 << 26) - 1, 1 << 26, INT32_MAX, -1, INT32_MIN};
  for (unsigned i = 0; i < 8; ++i)
    for (unsigned j = 0; j < 8; ++j) {
      const int valid = seqs[i] >= 0 && seqs[i] < 1 << 22 && width[j] >= 0 && width[j] < 1 << 26;
      const int before = stub_launches();
      CHECK((emb_history_step_workspace_bytes(h, kv, seqs[i], width[j]) > 0) == valid);
      EXPECT(emb_history_step(h, kv, seqs[i], FAKE(1), 512, 64, FAKE(2), 512, 64, FAKE(3), FAKE(4), width[j], FAKE(5),
                              seqs[i] ? FAKE(6) : NULL, SIZE_MAX, NULL, NULL), valid ? EMB_OK : EMB_E_INVAL);
      CHECK(stub_launches() - before == (valid && seqs[i] > 0));
    }
  EXPECT(emb_history_step(h, kv, 4, FAKE(1), 512, 64, FAKE(2), 512, 64, FAKE(3), FAKE(4), 8, FAKE(5), NULL, 1 << 20, NULL,
                          NULL), EMB_E_INVAL);
  EXPECT(emb_history_step(h, kv, 4, FAKE(1), 512, 64, FAKE(2), 512, 64, FAKE(3), FAKE(4), 8, FAKE(5), FAKE(6), 8, NULL,
                          NULL), EMB_E_WORKSPACE);
  emb_destroy_kv(kv);
  emb_destroy_history(h);
  return 0;
}

static int rows(void) {
  const int64_t n[] = {0, 1, 300, (1ll << 31) - 1, 1ll << 31, -1, INT64_MAX, INT64_MIN};
  const int32_t dims[] = {1, 7, EMB_MAX_ROW_DIM, EMB_MAX_ROW_DIM + 1, 0, -1, INT32_MAX, INT32_MIN};
  for (unsigned i = 0; i < 8; ++i)
    for (unsigned j = 0; j < 8; ++j) {
      const int fits = n[i] >= 0 && n[i] < 1ll << 31 && dims[j] >= 1;
      const int valid = fits && dims[j] <= EMB_MAX_ROW_DIM;
      const int64_t s = dims[j] > 0 ? dims[j] : 1;
      EXPECT(emb_layer_norm(n[i], dims[j], FAKE(1), EMB_BF16, s, FAKE(2), EMB_BF16, s, NULL, NULL, 0.f, NULL),
             valid ? EMB_OK : EMB_E_INVAL);
      CHECK(emb_layer_norm_workspace_bytes(n[i], dims[j]) ==
            (valid ? (size_t)(n[i] < 256 ? n[i] : 256) * 2 * dims[j] * 4 : 0));
      EXPECT(emb_layer_norm_backward(n[i], dims[j], FAKE(1), EMB_F32, s, FAKE(2), EMB_F16, s, FAKE(3), s, NULL, 1.f,
                                     FAKE(4), SIZE_MAX, NULL, NULL, NULL), valid ? EMB_OK : EMB_E_INVAL);
      const double p[] = {0.0, DBL_MIN, 0.1, 1.0 - 0x1p-53, 1.0, -DBL_MIN, 1.0 + 0x1p-52, INFINITY, NAN};
      for (unsigned k = 0; k < 9; ++k)
        EXPECT(emb_dropout(n[i], dims[j], EMB_F32, FAKE(1), s, NULL, 0, FAKE(2), s, p[k], UINT64_MAX, NULL, NULL),
               fits && p[k] >= 0 && p[k] <= 1 ? EMB_OK : EMB_E_INVAL);
    }
  return 0;
}

int main(void) {
  if (descriptors() || attention() || step() || rows()) return 1;
  printf("layer harness ok: %d checks\n", g_checks);
  return 0;
}
