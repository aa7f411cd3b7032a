/* Host-only driver for the C-ABI layer of the delta rule and the norms, linked
 * against their host code built with AddressSanitizer and
 * UndefinedBehaviorSanitizer and against launchers that only count. Calls that
 * have to be refused reach no launcher; those at the largest sizes the header
 * allows do, with every part of the workspace in place. Exit status 0 and "ok"
 * on success. */
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "retention.h"

extern int launches;
static int failures = 0;

static void expect(const char *what, long long got, long long want) {
  if (got != want) {
    printf("FAIL %s: %lld, want %lld\n", what, got, want);
    ++failures;
  }
}
static void refused(const char *what, int got, int want) {
  expect(what, got, want);
  expect("no launch", launches, 0);
  launches = 0;
}
static void launched(const char *what, int got) {
  expect(what, got, RET_OK);
  expect("one launch", launches, 1);
  launches = 0;
}

/* fake device addresses, 2^48 apart: validation only compares and aligns them */
#define A(i) ((void *)(uintptr_t)((uint64_t)(i) << 48))
#define F(i) ((float *)A(i))

static ret_delta_desc_t delta(int b, int n, int hk, int h, int d, int dtype) {
  ret_delta_desc_t r = {b, n, hk, h, d, d, dtype, 1.0f};
  return r;
}
static int fwd(const ret_delta_desc_t *d, const int32_t *cu, int64_t total, void *ws, size_t bytes) {
  return retention_delta_fwd(d, cu, total, A(1), A(2), A(3), F(4), F(5), A(6), F(7), F(7), ws, bytes, NULL);
}
static int bwd(const ret_delta_desc_t *d, const int32_t *cu, int64_t total, float *dsi, void *ws, size_t bytes) {
  return retention_delta_bwd(d, cu, total, A(1), A(2), A(3), F(4), F(5), A(6), F(7), F(8), A(9), A(10), A(11), F(12),
                             F(13), dsi, ws, bytes, NULL);
}
static int step(const ret_delta_desc_t *d, const int32_t *slots, int64_t n) {
  return retention_delta_step(d, A(1), A(2), A(3), F(4), F(5), A(6), F(7), slots, n, NULL);
}

static void delta_rule(void) {
  const int32_t *cu = (const int32_t *)A(20);
  /* the largest sizes: heads, batch of one-token sequences, tokens */
  const ret_delta_desc_t large[] = {delta(8191, 64, 1, 128, 256, RET_BF16), delta(1, 536870848, 1, 1, 64, RET_F32),
                                    delta(1048575, 1, 1, 1, 256, RET_F32), delta(2, 8192, 16, 128, 256, RET_BF16)};
  for (int i = 0; i < 4; ++i) {
    const ret_delta_desc_t *d = large + i;
    const size_t f = retention_delta_workspace_bytes(d, 0, 0), b = retention_delta_bwd_workspace_bytes(d, 0, 0);
    if (!(f > 0 && b > f)) expect("workspace sizes", i, -1);
    launched("fwd", fwd(d, NULL, 0, A(15), f));
    launched("bwd", bwd(d, NULL, 0, F(14), A(15), b));
    refused("fwd short", fwd(d, NULL, 0, A(15), f - 1), RET_ERR_WORKSPACE);
    refused("bwd short", bwd(d, NULL, 0, F(14), A(15), b - 1), RET_ERR_WORKSPACE);
    const int64_t all = (int64_t)d->batch * d->seqlen, totals[] = {0, 1, all};
    for (int j = 0; j < 3; ++j) {
      launched("packed fwd",
               fwd(d, cu, totals[j], A(15), retention_delta_workspace_bytes(d, 1, totals[j])));
      launched("packed bwd",
               bwd(d, cu, totals[j], F(14), A(15), retention_delta_bwd_workspace_bytes(d, 1, totals[j])));
    }
    refused("packed past the batch", fwd(d, cu, all + 1, A(15), SIZE_MAX), RET_ERR_SHAPE);
    refused("packed below zero", bwd(d, cu, INT64_MIN, F(14), A(15), SIZE_MAX), RET_ERR_SHAPE);
    refused("packed far past", fwd(d, cu, INT64_MAX, A(15), SIZE_MAX), RET_ERR_SHAPE);
  }
  /* whatever the descriptor holds */
  const int values[] = {INT_MIN, -1, 0, 1, 2, 63, 64, 65, 128, 129, 256, 1 << 20, 1 << 23, INT_MAX - 63, INT_MAX};
  const int n = (int)(sizeof values / sizeof *values);
  for (int a = 0; a < n; ++a)
    for (int b = 0; b < n; ++b)
      for (int c = 0; c < n; ++c) {
        ret_delta_desc_t d = delta(values[a], values[b], 1, values[c], 128, RET_BF16);
        const size_t f = retention_delta_workspace_bytes(&d, 0, 0);
        const int got = fwd(&d, NULL, 0, A(15), f);
        if (got != RET_OK && got != RET_ERR_SHAPE) expect("descriptor", got, RET_ERR_SHAPE);
        expect("size and status agree", f > 0, got == RET_OK);
        ret_delta_desc_t k = delta(1, 64, values[a], values[b], values[c], values[c]);
        if (fwd(&k, NULL, 0, NULL, 0) == RET_OK) expect("no workspace", 0, 1);
        d.seqlen = 1;
        step(&d, (const int32_t *)A(16), values[b]);
      }
  launches = 0;
  ret_delta_desc_t d = delta(2, 100, 2, 4, 128, RET_BF16);
  refused("NULL desc", fwd(NULL, NULL, 0, A(15), SIZE_MAX), RET_ERR_NULL);
  refused("NULL desc", bwd(NULL, NULL, 0, NULL, A(15), SIZE_MAX), RET_ERR_NULL);
  refused("state_in without its gradient", bwd(&d, NULL, 0, NULL, A(15), SIZE_MAX), RET_ERR_NULL);
  refused("workspace over q", fwd(&d, NULL, 0, A(1), SIZE_MAX), RET_ERR_ALIAS);
  refused("bounds inside the workspace", fwd(&d, (const int32_t *)A(15), 10, A(15), SIZE_MAX), RET_ERR_ALIAS);
  d.scale = NAN;
  refused("scale", fwd(&d, NULL, 0, A(15), SIZE_MAX), RET_ERR_ARG);
  d = delta(3, 1, 2, 4, 64, RET_F32);
  launched("step", step(&d, NULL, 3));
  launched("step, largest pool", step(&d, (const int32_t *)A(16), INT32_MAX));
  refused("step pool", step(&d, NULL, 4), RET_ERR_SHAPE);
  refused("step pool", step(&d, (const int32_t *)A(16), INT64_MAX), RET_ERR_SHAPE);
  refused("step pool", step(&d, (const int32_t *)A(16), INT64_MIN), RET_ERR_SHAPE);
  refused("step NULL", step(NULL, NULL, 1), RET_ERR_NULL);
}

static void norms(void) {
  const int64_t rows[] = {INT64_MIN, -1, 0, 1, 65, INT32_MAX, (int64_t)INT32_MAX + 1, INT64_MAX};
  const int widths[] = {INT_MIN, 0, 1, 7, 2048, 4100, 16384, 16385, INT_MAX};
  for (int a = 0; a < 8; ++a)
    for (int b = 0; b < 9; ++b)
      for (int dtype = -1; dtype <= 2; ++dtype) {
        ret_norm_desc_t d = {rows[a], widths[b], dtype, 1, 1e-5f};
        const int ok = rows[a] >= 0 && rows[a] <= INT32_MAX && widths[b] >= 1 && widths[b] <= 16384 &&
                       (dtype == 0 || dtype == 1);
        const size_t h = retention_head_norm_bwd_workspace_bytes(&d), r = retention_residual_norm_bwd_workspace_bytes(&d);
        expect("sizes", h > 0 && r == 3 * h, ok);
        const int got[] = {
            retention_head_norm_fwd(&d, A(1), F(2), A(3), A(4), NULL),
            retention_head_norm_bwd(&d, A(1), F(2), A(3), A(4), A(5), F(6), A(7), A(8), h, NULL),
            retention_residual_norm_fwd(&d, 1.0f, A(1), A(2), F(3), F(4), F(5), A(6), A(1), NULL),
            retention_residual_norm_bwd(&d, 1.0f, A(1), A(2), F(3), F(4), F(5), A(6), A(7), A(8), A(9), F(10), F(11),
                                        F(12), A(13), r, NULL)};
        for (int i = 0; i < 4; ++i) expect("norm status", got[i] == RET_OK, ok);
        expect("norm launches", launches, !ok ? 0 : rows[a] ? 4 : 2);
        launches = 0;
      }
  ret_norm_desc_t d = {64, 256, RET_BF16, 0, 1e-5f};
  const size_t h = retention_head_norm_bwd_workspace_bytes(&d);
  refused("short", retention_head_norm_bwd(&d, A(1), F(2), NULL, A(4), A(5), F(6), NULL, A(8), h - 1, NULL),
          RET_ERR_WORKSPACE);
  refused("weight without its gradient",
          retention_head_norm_bwd(&d, A(1), F(2), NULL, A(4), A(5), NULL, NULL, A(8), h, NULL), RET_ERR_NULL);
  refused("skip", retention_residual_norm_fwd(&d, INFINITY, A(1), A(2), F(3), NULL, NULL, A(6), A(7), NULL), RET_ERR_ARG);
  refused("over the input", retention_head_norm_fwd(&d, A(1), NULL, NULL, (char *)A(1) + 16, NULL), RET_ERR_ALIAS);
  refused("NULL desc", retention_head_norm_fwd(NULL, A(1), NULL, NULL, A(2), NULL), RET_ERR_NULL);
}

int main(void) {
  delta_rule();
  norms();
  if (failures) return 1;
  printf("ok\n");
  return 0;
}
