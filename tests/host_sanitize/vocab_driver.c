/*
 * Host-side check of the vocabulary layer's and the optimizer's calls of
 * qlora.h under AddressSanitizer and UndefinedBehaviorSanitizer: size queries
 * up to the edges of the index ranges, and arguments that validation must turn
 * into a status before any device work. Nothing here may launch a kernel; exit
 * status 0 when every status matches.
 */
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "qlora.h"

static int failures = 0, checks = 0;

static void expect(int got, int want, const char* what) {
  ++checks;
  if (got != want) {
    ++failures;
    printf("FAIL %s: status %d, expected %d\n", what, got, want);
  }
}

/* Stand-ins for device buffers, compared and never dereferenced. */
static _Alignas(256) unsigned char arena[1 << 16];
#define P(off) ((void*)(arena + (off)))

static qlora_linear layer(int K, int N, int r, int fmt) {
  qlora_linear L;
  memset(&L, 0, sizeof L);
  L.K = K; L.N = N; L.r = r; L.alpha = 16.f; L.fmt = fmt;
  L.codes = P(0); L.scales = P(256);
  L.A = r > 0 ? (const float*)P(512) : NULL;
  L.B = r > 0 ? (const float*)P(768) : NULL;
  return L;
}

int main(void) {
  static const struct { int K, N, r, fmt, vocab, M, dt, embed_bwd, xent; } sizes[] = {
      {16, 16, 1, QLORA_W8, 1, 1, QLORA_F32, 0, 0},
      {2048, 256000, 8, QLORA_W8, 256000, 8192, QLORA_BF16, 0, 0},
      {768, 50272, 32, QLORA_W8, 50257, 1 << 20, QLORA_F32, 0, 0},
      {768, 50272, 32, QLORA_W8, 50257, (1 << 20) + 1, QLORA_F32, QLORA_ERANGE, 0},
      {4096, 32000, 8, QLORA_W4G128, 32000, 4096, QLORA_BF16, 0, 0},
      {16384, 131056, 32, QLORA_W4G128, 131056, 131071, QLORA_BF16, 0, 0},
      {16, 134217712, 32, QLORA_W8, 134217712, 1, QLORA_F32, 0, 0},
      {16, 134217712, 32, QLORA_W8, 134217712, 1024, QLORA_F32, 0, 0},
      {16, 134217712, 32, QLORA_W8, 134217712, 1025, QLORA_F32, 0, QLORA_ERANGE},
      {16, 134217728, 32, QLORA_W8, 1, 1, QLORA_F32, QLORA_ERANGE, QLORA_ERANGE},
      {16, 16, 32, QLORA_W8, 16, 1 << 24, QLORA_F32, QLORA_ERANGE, 0},
      {16, 16, 32, QLORA_W8, 16, 134217727, QLORA_F32, QLORA_ERANGE, QLORA_ERANGE},
      {16, 16, 32, QLORA_W8, 16, INT_MAX, QLORA_F32, QLORA_ERANGE, QLORA_ERANGE},
      {INT_MAX - 15, 16, 1, QLORA_W8, 16, 1, QLORA_F32, QLORA_ERANGE, QLORA_ERANGE},
      {134217712, 16, 32, QLORA_W8, 16, 1, QLORA_F32, QLORA_ERANGE, QLORA_ERANGE},
      {1 << 23, 16, 32, QLORA_W8, 16, 1, QLORA_F32, 0, QLORA_EUNSUPPORTED},
      {132112, 16, 32, QLORA_W8, 16, 1, QLORA_F32, 0, QLORA_EUNSUPPORTED},
      {16, 16, INT_MAX, QLORA_W8, 16, 1, QLORA_F32, QLORA_EINVAL, QLORA_EINVAL},
      {16, 16, 1, QLORA_W8, INT_MAX, 1, QLORA_F32, QLORA_EINVAL, QLORA_EINVAL},
      {16, 16, 1, QLORA_W8, INT_MIN, 1, QLORA_F32, QLORA_EINVAL, QLORA_EINVAL},
      {16, 16, 1, QLORA_W8, 16, INT_MIN, QLORA_F32, QLORA_EINVAL, QLORA_EINVAL},
      {16, 16, 1, INT_MAX, 16, 1, QLORA_F32, QLORA_EINVAL, QLORA_EINVAL},
      {INT_MIN, INT_MIN, 1, QLORA_W8, 16, 1, QLORA_F32, QLORA_EINVAL, QLORA_EINVAL},
  };
  size_t n = 0;
  for (size_t i = 0; i < sizeof sizes / sizeof sizes[0]; ++i) {
    const qlora_linear L = layer(sizes[i].K, sizes[i].N, sizes[i].r, sizes[i].fmt);
    expect(qlora_embed_bwd_workspace(&L, sizes[i].vocab, sizes[i].M, sizes[i].dt, &n), sizes[i].embed_bwd,
           "embed_bwd_workspace");
    expect(qlora_xent_fwd_workspace(&L, sizes[i].vocab, sizes[i].M, sizes[i].dt, &n), sizes[i].xent,
           "xent_fwd_workspace");
    expect(qlora_xent_bwd_workspace(&L, sizes[i].vocab, sizes[i].M, sizes[i].dt, &n), sizes[i].xent,
           "xent_bwd_workspace");
  }
  for (int r = 0; r < 8; r += 4) {
    const qlora_linear L = layer(64, 64, r, QLORA_W8);
    const int M = 3;
    size_t need = 0;
    expect(qlora_embed(&L, 60, M, QLORA_F32, P(1024), QLORA_I64, 1.f, P(0), NULL), QLORA_EINVAL, "embed overlap");
    expect(qlora_embed(&L, 60, M, QLORA_F32, P(1028), QLORA_I64, 1.f, P(4096), NULL), QLORA_EINVAL, "embed tokens");
    expect(qlora_embed(&L, 60, M, QLORA_F32, P(1024), INT_MAX, 1.f, P(4096), NULL), QLORA_EINVAL, "embed itype");
    expect(qlora_xent_fwd_workspace(&L, 60, M, QLORA_F32, &need), QLORA_OK, "xent_fwd_workspace");
    expect(qlora_xent_fwd(&L, 60, M, QLORA_F32, P(2048), P(1024), QLORA_I64, P(3072), P(3328), NULL, P(8192), need - 1,
                          NULL), QLORA_EWORKSPACE, "xent_fwd workspace");
    expect(qlora_xent_fwd(&L, 60, M, QLORA_F32, P(2048), P(1024), QLORA_I64, P(3072), P(3072), NULL, P(8192), need,
                          NULL), QLORA_EINVAL, "xent_fwd overlap");
    expect(qlora_xent_bwd_workspace(&L, 60, M, QLORA_F32, &need), QLORA_OK, "xent_bwd_workspace");
    expect(qlora_xent_bwd(&L, 60, M, QLORA_F32, P(2048), P(1024), QLORA_I64, P(3072), P(3328), NULL, P(2048),
                          r ? P(4096) : NULL, r ? P(6144) : NULL, P(8192), need, NULL), QLORA_EINVAL, "xent_bwd overlap");
    expect(qlora_xent_bwd(&L, 60, M, QLORA_F32, P(2048), P(1024), QLORA_I64, P(3072), P(3328), NULL, P(3584),
                          r ? P(4608) : NULL, r ? P(6144) : NULL, P(8192), need - 1, NULL), QLORA_EWORKSPACE,
           "xent_bwd workspace");
    if (r > 0) {
      expect(qlora_embed_bwd_workspace(&L, 60, M, QLORA_F32, &need), QLORA_OK, "embed_bwd_workspace");
      expect(qlora_embed_bwd(&L, 60, M, QLORA_F32, P(1024), QLORA_I32, 1.f, P(2048), 0, P(4608), P(4608), P(8192), need,
                             NULL), QLORA_EINVAL, "embed_bwd overlap");
      expect(qlora_embed_bwd(&L, 60, M, QLORA_F32, P(1024), QLORA_I32, 1.f, P(2048), 1, P(4608), P(6144), P(8192),
                             need - 1, NULL), QLORA_EWORKSPACE, "embed_bwd workspace");
    }
  }
  expect(qlora_embed(NULL, 1, 1, QLORA_F32, P(0), QLORA_I32, 1.f, P(256), NULL), QLORA_EINVAL, "no layer");
  expect(qlora_xent_fwd_workspace(NULL, 1, 1, QLORA_F32, &n), QLORA_EINVAL, "no layer");
  expect(qlora_xent_bwd_workspace(NULL, 1, 1, QLORA_F32, &n), QLORA_EINVAL, "no layer");
  expect(qlora_embed_bwd_workspace(NULL, 1, 1, QLORA_F32, &n), QLORA_EINVAL, "no layer");

  /* the optimizer: many tensors, of the smallest and the largest size */
  static qlora_adamw_item items[1000];
  for (int i = 0; i < 1000; ++i) {
    items[i].p = P(0); items[i].g = P(4096); items[i].m = P(8192); items[i].v = P(12288);
    items[i].n = i % 3 == 0 ? (int64_t)1 << 30 : i + 1;
  }
  expect(qlora_adamw_workspace(items, 1000, &n), QLORA_OK, "adamw_workspace");
  items[999].n = INT64_MAX;
  expect(qlora_adamw_workspace(items, 1000, &n), QLORA_ERANGE, "adamw_workspace elements");
  items[999].n = INT64_MIN;
  expect(qlora_adamw_workspace(items, 1000, &n), QLORA_EINVAL, "adamw_workspace elements");
  expect(qlora_adamw_workspace(items, INT_MIN, &n), QLORA_EINVAL, "adamw_workspace count");
  qlora_adamw_config c;
  memset(&c, 0, sizeof c);
  c.lr = 1e-3; c.beta1 = 0.9; c.beta2 = 0.999; c.eps = 1e-6; c.step = (int32_t*)P(256);
  items[0].n = 64;
  expect(qlora_adamw(&c, items, 1, P(16384), 0, NULL), QLORA_EWORKSPACE, "adamw workspace");
  c.step = (int32_t*)P(252);                       /* p holds the bytes up to 255 */
  expect(qlora_adamw(&c, items, 1, P(16384), 1 << 12, NULL), QLORA_EINVAL, "adamw overlap");
  c.step = (int32_t*)P(256);
  c.lr = NAN;
  expect(qlora_adamw(&c, items, 1, P(16384), 1 << 12, NULL), QLORA_EINVAL, "adamw learning rate");
  c.lr = 1e300;
  expect(qlora_adamw(&c, items, 1, P(16384), 1 << 12, NULL), QLORA_EINVAL, "adamw learning rate");
  c.lr = 0; c.eps = 1e-300;
  expect(qlora_adamw(&c, items, 1, P(16384), 1 << 12, NULL), QLORA_EINVAL, "adamw eps");
  expect(qlora_moment_read(P(0), P(256), INT64_MAX, QLORA_MOMENT1, QLORA_F32, P(1024), NULL), QLORA_ERANGE, "moment");
  expect(qlora_moment_read(P(0), P(256), INT64_MIN, QLORA_MOMENT1, QLORA_F32, P(1024), NULL), QLORA_EINVAL, "moment");
  expect(qlora_moment_write(P(0), 64, QLORA_MOMENT2, QLORA_BF16, P(112), P(1024), NULL), QLORA_EINVAL, "moment overlap");
  expect(qlora_moment_write(P(0), 64, INT_MAX, QLORA_BF16, P(512), P(1024), NULL), QLORA_EINVAL, "moment kind");
  printf("%d checks, %d failures\n", checks, failures);
  return failures != 0;
}
