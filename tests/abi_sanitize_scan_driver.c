/* Host-only driver for the C-ABI layer of the recurrence, the convolution and the
 * cache of parked states, linked against their host code built with
 * AddressSanitizer and UndefinedBehaviorSanitizer and against launchers that only
 * count. Calls that have to be refused reach no launcher; those at the largest
 * sizes the header allows do. Exit status 0 and "ok" on success. */
#include <limits.h>
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
static void launched(const char *what, int got, int n) {
  expect(what, got, RET_OK);
  expect(what, launches, n);
  launches = 0;
}

/* fake device addresses, 2^48 apart: validation only compares and aligns them */
#define A(i) ((void *)(uintptr_t)((uint64_t)(i) << 48))
#define F(i) ((float *)A(i))
#define I(i) ((int32_t *)A(i))

static ret_scan_desc_t scan(int b, int n, int w, int dtype) {
  ret_scan_desc_t d = {b, n, w, dtype, 1, 0, 0, 0, 0};
  return d;
}
static ret_conv_desc_t conv(int b, int n, int w, int taps, int dtype) {
  ret_conv_desc_t d = {b, n, w, taps, dtype, 1, 0};
  return d;
}
static int sf(const ret_scan_desc_t *d, const int32_t *cu, int64_t total, void *ws, size_t n) {
  return retention_scan_fwd(d, cu, total, A(1), A(2), F(3), A(4), A(5), F(6), F(6), F(7), ws, n, NULL);
}
static int sb(const ret_scan_desc_t *d, const int32_t *cu, int64_t total, const float *kept, void *ws, size_t n) {
  return retention_scan_bwd(d, cu, total, A(1), A(2), F(3), A(4), A(5), F(6), F(7), kept, A(9), A(10), F(11), A(12), F(13),
                            ws, n, NULL);
}
static int cf(const ret_conv_desc_t *d, const int32_t *cu, int64_t total, void *ws, size_t n) {
  return retention_conv_fwd(d, cu, total, A(1), F(2), F(3), A(4), A(5), A(5), ws, n, NULL);
}
static int cb(const ret_conv_desc_t *d, const int32_t *cu, int64_t total, void *ws, size_t n) {
  return retention_conv_bwd(d, cu, total, A(1), F(2), F(3), A(4), A(5), A(6), A(7), F(8), F(9), A(10), ws, n, NULL);
}

static void sequences(void) {
  const int32_t *cu = I(20);
  const int64_t most = (int64_t)INT32_MAX - 65536;
  const ret_scan_desc_t large[] = {scan(1, 536870656, 64, RET_BF16), scan(2097151, 128, 1, RET_F32),
                                   scan(1, 262144, 65536, RET_F32), scan(3, 1, 1, RET_BF16), scan(1 << 20, 1, 64, RET_F32)};
  for (int i = 0; i < 5; ++i) {
    const ret_scan_desc_t *d = large + i;
    const ret_conv_desc_t c = conv(d->batch, d->seqlen, d->width, 2 + i % 3, d->dtype);
    const int64_t all = (int64_t)d->batch * d->seqlen, totals[] = {0, 1, all};
    const size_t f = retention_scan_workspace_bytes(d, 0, 0), b = retention_scan_bwd_workspace_bytes(d, 0, 0, 1),
                 own = retention_scan_bwd_workspace_bytes(d, 0, 0, 0), cw = retention_conv_bwd_workspace_bytes(&c, 0, 0);
    launched("scan fwd", sf(d, NULL, 0, A(15), f), 1);
    launched("scan bwd", sb(d, NULL, 0, F(8), A(15), b), 1);
    launched("scan bwd of its own states", sb(d, NULL, 0, NULL, A(15), own), 2);
    refused("short", sf(d, NULL, 0, A(15), f - 1), RET_ERR_WORKSPACE);
    refused("short", sb(d, NULL, 0, F(8), A(15), b - 1), RET_ERR_WORKSPACE);
    refused("short", sb(d, NULL, 0, NULL, A(15), own - 1), RET_ERR_WORKSPACE);
    launched("conv fwd", cf(&c, NULL, 0, NULL, 0), 1);
    launched("conv bwd", cb(&c, NULL, 0, A(15), cw), 1);
    refused("short", cb(&c, NULL, 0, A(15), cw - 1), RET_ERR_WORKSPACE);
    for (int j = 0; j < 3; ++j) {
      const int64_t t = totals[j];
      launched("packed scan fwd", sf(d, cu, t, A(15), retention_scan_workspace_bytes(d, 1, t)), 1);
      launched("packed scan bwd", sb(d, cu, t, NULL, A(15), retention_scan_bwd_workspace_bytes(d, 1, t, 0)), 2);
      launched("packed conv fwd", cf(&c, cu, t, A(15), retention_conv_workspace_bytes(&c, 1, t)), 1);
      launched("packed conv bwd", cb(&c, cu, t, A(15), retention_conv_bwd_workspace_bytes(&c, 1, t)), 1);
    }
    refused("too many tokens", sf(d, cu, most + 1, A(15), SIZE_MAX), RET_ERR_SHAPE);
    refused("below zero", sb(d, cu, INT64_MIN, NULL, A(15), SIZE_MAX), RET_ERR_SHAPE);
    refused("far past", cf(&c, cu, INT64_MAX, A(15), SIZE_MAX), RET_ERR_SHAPE);
    refused("far past", cb(&c, cu, INT64_MAX, A(15), SIZE_MAX), RET_ERR_SHAPE);
  }
  /* whatever the descriptor holds */
  const int v[] = {INT_MIN, -1, 0, 1, 2, 63, 64, 65, 128, 256, 257, 513, 65536, 65537, 1 << 20, INT_MAX - 65536, INT_MAX};
  const int64_t st[] = {INT64_MIN, -1, 0, 1, 64, 1 << 20, 1 << 22, INT32_MAX, (int64_t)1 << 40, INT64_MAX};
  for (int a = 0; a < 17; ++a)
    for (int b = 0; b < 17; ++b)
      for (int c = 0; c < 17; ++c)
        for (int s = 0; s < 10; ++s) {
          ret_scan_desc_t d = scan(v[a], v[b], v[c], s & 1);
          d.x_stride = st[s];
          d.gate_stride = st[(s + a) % 10];
          const size_t f = retention_scan_workspace_bytes(&d, 0, 0);
          const int got = sf(&d, NULL, 0, A(15), f);
          if (got != RET_OK && got != RET_ERR_SHAPE && got != RET_ERR_ALIAS) expect("descriptor", got, RET_ERR_SHAPE);
          expect("size and status agree", f > 0, got == RET_OK || got == RET_ERR_ALIAS);
          ret_conv_desc_t k = conv(v[a], v[b], v[c], 4, s & 1);
          k.x_stride = st[s];
          const size_t cw = retention_conv_bwd_workspace_bytes(&k, 0, 0);
          const int gc = cb(&k, NULL, 0, A(15), cw);
          expect("size and status agree", cw > 0, gc == RET_OK || gc == RET_ERR_ALIAS);
          if (sf(&d, NULL, 0, NULL, 0) == RET_OK) expect("no workspace", 0, 1);
          d.seqlen = k.seqlen = 1;
          retention_scan_step(&d, A(1), A(2), NULL, A(4), A(5), F(6), I(7), st[s], NULL);
          retention_conv_step(&k, A(1), F(2), NULL, A(4), A(5), I(6), st[s], NULL);
        }
  launches = 0;
  ret_scan_desc_t d = scan(2, 1000, 64, RET_BF16);
  refused("NULL desc", sf(NULL, NULL, 0, A(15), SIZE_MAX), RET_ERR_NULL);
  refused("NULL desc", sb(NULL, NULL, 0, NULL, A(15), SIZE_MAX), RET_ERR_NULL);
  refused("NULL desc", cf(NULL, NULL, 0, A(15), SIZE_MAX), RET_ERR_NULL);
  refused("workspace over x", sf(&d, NULL, 0, A(1), SIZE_MAX), RET_ERR_ALIAS);
  refused("bounds inside the workspace", sf(&d, I(15), 10, A(15), SIZE_MAX), RET_ERR_ALIAS);
  refused("kept inside the workspace", sb(&d, NULL, 0, F(15), A(15), SIZE_MAX), RET_ERR_ALIAS);
  d = scan(3, 1, 64, RET_F32);
  launched("step, largest pool", retention_scan_step(&d, A(1), A(2), NULL, NULL, A(5), F(6), I(7), INT32_MAX, NULL), 1);
  refused("step pool", retention_scan_step(&d, A(1), A(2), NULL, NULL, A(5), F(6), I(7), INT64_MAX, NULL), RET_ERR_SHAPE);
  refused("step NULL", retention_scan_step(NULL, A(1), A(2), NULL, NULL, A(5), F(6), NULL, 1, NULL), RET_ERR_NULL);
}

static void cache(void) {
  const int64_t v[] = {INT64_MIN, -1, 0, 1, 63, 64, 65, 1 << 20, (int64_t)1 << 33, INT32_MAX, (int64_t)1 << 40, INT64_MAX};
  const int b[] = {INT_MIN, 0, 1, 64, 65535, 65536, INT_MAX};
  for (int i = 0; i < 12; ++i)
    for (int j = 0; j < 12; ++j)
      for (int k = 0; k < 7; ++k) {
        const ret_state_cache_desc_t d = {b[k], 0, v[i], v[j], v[(i + j) % 12]};
        const int w = retention_state_cache_write(&d, F(1), A(2), F(100), I(200), I(201), NULL);
        const int r = retention_state_cache_read(&d, A(2), F(100), F(1), I(200), I(201), NULL);
        if (w != RET_OK && w != RET_ERR_SHAPE && w != RET_ERR_ALIAS) expect("cache", w, RET_ERR_SHAPE);
        if (r != RET_OK && r != RET_ERR_SHAPE && r != RET_ERR_ALIAS) expect("cache", r, RET_ERR_SHAPE);
        expect("cache launches", launches, (w == RET_OK) + (r == RET_OK));
        launches = 0;
      }
  refused("NULL desc", retention_state_cache_write(NULL, F(1), A(2), F(3), I(4), NULL, NULL), RET_ERR_NULL);
}

int main(void) {
  sequences();
  cache();
  if (failures) return 1;
  printf("ok\n");
  return 0;
}
