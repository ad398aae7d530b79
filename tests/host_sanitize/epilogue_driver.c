/*
 * Host-side check of the epilogue and checkpoint calls of qlora.h under
 * AddressSanitizer and UndefinedBehaviorSanitizer: size queries up to the edge
 * of the index range, and arguments that validation must turn into a status
 * before any device work. Nothing here may launch a kernel; exit status 0
 * when every status matches.
 */
#include <limits.h>
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
  L.codes = P(0); L.scales = P(256); L.A = (const float*)P(512); L.B = (const float*)P(768);
  return L;
}

int main(void) {
  size_t cb = 0, sb = 0;
  static const int sizes[][4] = {
      /* M, C, form, status */
      {1, 16, 0, 0}, {1, 16, 1, 0}, {0, 16, 0, 1}, {-1, 16, 1, 1}, {INT_MIN, 16, 0, 1}, {1, 0, 0, 1},
      {1, -16, 0, 1}, {1, 17, 1, 1}, {INT_MAX, 16, 0, 4}, {1, INT_MAX - 15, 0, 0}, {1, INT_MAX - 15, 1, 0}, {1, 1 << 30, 0, 0}, {2, 1 << 30, 1, 4},
      {134217727, 16, 1, 0}, {134217728, 16, 1, 4}, {5, 80, 2, 1}, {5, 80, -1, 1}, {5, 80, INT_MAX, 1},
  };
  for (size_t i = 0; i < sizeof sizes / sizeof sizes[0]; ++i)
    expect(qlora_ckpt_bytes(sizes[i][0], sizes[i][1], sizes[i][2], &cb, &sb), sizes[i][3], "ckpt_bytes");
  expect(qlora_ckpt_bytes(1, 16, 0, NULL, &sb), QLORA_EINVAL, "ckpt_bytes null");
  expect(qlora_ckpt_bytes(1, 16, 0, &cb, NULL), QLORA_EINVAL, "ckpt_bytes null");
  static const int acts[][3] = {
      /* M, N, status */
      {1, 16, 0}, {4096, 2304, 0}, {134217727, 16, 0}, {134217728, 16, 4}, {1, INT_MAX - 15, 0},
      {0, 16, 1}, {1, 24, 1}, {INT_MIN, INT_MIN, 1}, {INT_MAX, INT_MAX - 15, 4},
  };
  for (size_t i = 0; i < sizeof acts / sizeof acts[0]; ++i)
    expect(qlora_act_bwd_workspace(acts[i][0], acts[i][1], &cb), acts[i][2], "act_bwd_workspace");

  static const int shapes[][5] = {
      {64, 256, 256, 4, QLORA_W8}, {1, 2048, 16384, 8, QLORA_W8}, {8, 16, 16, 32, QLORA_W8},
      {1001, 784, 1024, 8, QLORA_W8}, {512, 16384, 2048, 8, QLORA_W8O}, {2048, 4096, 4096, 4, QLORA_W4G128},
      {131071, 16384, 16, 1, QLORA_W8},
  };
  for (size_t i = 0; i < sizeof shapes / sizeof shapes[0]; ++i) {
    const int M = shapes[i][0], r = shapes[i][3];
    qlora_linear L = layer(shapes[i][1], shapes[i][2], r, shapes[i][4]);
    qlora_epilogue e;
    qlora_grad_epilogue g;
    size_t need = 0;
    memset(&e, 0, sizeof e);
    memset(&g, 0, sizeof g);
    expect(qlora_fwd_workspace(&L, M, QLORA_BF16, &need), QLORA_OK, "fwd_workspace");
    expect(qlora_fwd_epi(&L, M, QLORA_BF16, P(1024), NULL, P(2048), NULL, P(4096), need, NULL), QLORA_EINVAL,
           "fwd_epi without an epilogue");
    expect(qlora_fwd_epi(&L, M, QLORA_BF16, P(1024), &e, P(2048), NULL, P(4096), need - 1, NULL),
           QLORA_EWORKSPACE, "fwd_epi workspace");
    expect(qlora_fwd_ckpt(&L, M, QLORA_BF16, P(1024), P(1280), P(1536), &e, P(2048), P(4096), need - 1, NULL),
           QLORA_EWORKSPACE, "fwd_ckpt workspace");
    /* every buffer in one small arena: they overlap */
    expect(qlora_fwd_epi(&L, M, QLORA_BF16, P(1024), &e, P(1024), NULL, P(4096), need, NULL), QLORA_EINVAL,
           "fwd_epi overlap");
    expect(qlora_fwd_ckpt(&L, M, QLORA_BF16, P(1024), P(1280), P(1536), &e, P(1024), P(4096), need, NULL),
           QLORA_EINVAL, "fwd_ckpt overlap");
    e.act = INT_MIN;
    expect(qlora_fwd_epi(&L, M, QLORA_BF16, P(1024), &e, P(2048), NULL, P(4096), need, NULL), QLORA_EINVAL,
           "activation");
    expect(qlora_bwd_epi_workspace(&L, M, QLORA_BF16, &need), QLORA_OK, "bwd_epi_workspace");
    expect(qlora_bwd_epi_workspace(&L, 0, QLORA_BF16, &need), QLORA_EINVAL, "bwd_epi_workspace rows");
    expect(qlora_bwd_epi_workspace(&L, M, QLORA_BF16, NULL), QLORA_EINVAL, "bwd_epi_workspace null");
    expect(qlora_bwd_epi(&L, M, QLORA_BF16, NULL, P(1024), P(1280), P(1536), NULL, NULL, P(2048), P(2304),
                         P(2560), P(4096), need, NULL), QLORA_EINVAL, "bwd_epi without t");
    expect(qlora_bwd_epi(&L, M, QLORA_BF16, NULL, P(1024), P(1280), P(1536), P(1792), NULL, P(2048), P(2304),
                         P(2560), P(4096), need - 1, NULL), QLORA_EWORKSPACE, "bwd_epi workspace");
    expect(qlora_bwd_epi_partial(&L, M, QLORA_BF16, NULL, P(1024), P(1280), P(1536), P(1792), NULL, P(1024),
                                 P(4096), need, NULL), QLORA_EINVAL, "bwd_epi_partial overlap");
    g.act = INT_MAX;
    expect(qlora_bwd_epi(&L, M, QLORA_BF16, NULL, P(1024), P(1280), P(1536), P(1792), &g, P(2048), P(2304),
                         P(2560), P(4096), need, NULL), QLORA_EINVAL, "gradient activation");
  }
  expect(qlora_fwd_epi(NULL, 1, QLORA_BF16, P(0), NULL, P(0), NULL, P(0), 0, NULL), QLORA_EINVAL, "no layer");
  expect(qlora_fwd_ckpt(NULL, 1, QLORA_BF16, P(0), P(0), P(0), NULL, P(0), P(0), 0, NULL), QLORA_EINVAL, "no layer");
  expect(qlora_bwd_epi(NULL, 1, QLORA_BF16, P(0), NULL, NULL, P(0), P(0), NULL, P(0), P(0), P(0), P(0), 0, NULL),
         QLORA_EINVAL, "no layer");
  expect(qlora_ckpt_write(P(0), 1, 16, QLORA_F32, QLORA_C8G32, P(32), P(256), NULL), QLORA_EINVAL, "overlap");
  expect(qlora_ckpt_read(P(0), P(256), 1, 16, QLORA_C8G32, QLORA_F32, P(0), NULL), QLORA_EINVAL, "overlap");
  expect(qlora_act_bwd(2, 1, 16, QLORA_F32, P(0), P(256), NULL, NULL, P(16), NULL, NULL, 0, NULL), QLORA_EINVAL,
         "overlap");
  printf("%d checks, %d failures\n", checks, failures);
  return failures != 0;
}
