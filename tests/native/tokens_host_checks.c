/*
 * Host-side checks of the token operators' entry points, built and run by
 * tests/test_tokens_native.py against the regular library and against their
 * source with AddressSanitizer in its host code.  Only host logic runs:
 * workspace sizes, and argument errors that are reported before anything is
 * enqueued (no call here reaches a kernel launch; the pointers passed are never
 * dereferenced).
 */
#include <stdint.h>
#include <stdio.h>

#include "grz.h"

static int failures = 0;
#define REFUSED(call, want)                                                       \
  do {                                                                            \
    const int got = (call);                                                       \
    if (got != (want)) {                                                          \
      fprintf(stderr, "FAIL %s:%d: %s: %d\n", __FILE__, __LINE__, #call, got);    \
      ++failures;                                                                 \
    }                                                                             \
  } while (0)

static char* const A = (char*)0x100000;
static char* const B = (char*)0x20000000;
static char* const C = (char*)0x40000000;
static char* const D = (char*)0x60000000;
static char* const W = (char*)0x80000000;

static void embedding(void) {
  const int64_t limits[] = {INT64_MIN, -1, (int64_t)1 << 31, (int64_t)1 << 62, INT64_MAX};
  for (int i = 0; i < 5; ++i) {
    const int64_t v = limits[i];
    const int want = v < 0 ? GRZ_EINVAL : GRZ_ERANGE;
    REFUSED(dp_embed_lookup(A, GRZ_BF16, v, 8, 8, B, 64, 4, 1.0f, C, GRZ_BF16, 8, NULL), want);
    REFUSED(dp_embed_lookup(A, GRZ_BF16, 10, 8, 8, B, 64, v, 1.0f, C, GRZ_BF16, 8, NULL), want);
    REFUSED(dp_embed_lookup(A, GRZ_BF16, 10, v, v, B, 64, 4, 1.0f, C, GRZ_BF16, v, NULL), want);
    REFUSED(dp_embed_grad(A, GRZ_F32, 8, B, 32, v, 10, 8, 1.0f, 0, W, C, GRZ_F32, 8, NULL), want);
    REFUSED(dp_embed_grad(A, GRZ_F32, 8, B, 32, 4, v, 8, 1.0f, 0, W, C, GRZ_F32, 8, NULL), want);
    REFUSED(dp_embed_grad(A, GRZ_F32, v, B, 32, 4, 10, v, 1.0f, 0, W, C, GRZ_F32, v, NULL), want);
    if (dp_embed_grad_workspace(v, 10, 8) || dp_embed_grad_workspace(4, v, 8) ||
        dp_embed_grad_workspace(4, 10, v)) {
      fprintf(stderr, "FAIL workspace of a refused size\n");
      ++failures;
    }
  }
  REFUSED(dp_embed_lookup(A, GRZ_BF16, 10, 8, INT64_MAX, B, 64, 4, 1.0f, C, GRZ_BF16, 8, NULL),
          GRZ_ERANGE);
  REFUSED(dp_embed_grad(A, GRZ_F32, 8, B, 32, 4, 10, 8, 1.0f, 1, W, C, GRZ_F32, 8, NULL),
          GRZ_EINVAL);
  REFUSED(dp_embed_grad(A, GRZ_F32, 8, B, 32, 4, 10, 8, 1.0f, 0, W + 8, C, GRZ_F32, 8, NULL),
          GRZ_EALIGN);
  REFUSED(dp_embed_grad(A, GRZ_F32, 8, B, 32, 4, 10, 8, 1.0f, 0, A + 112, C, GRZ_F32, 8, NULL),
          GRZ_EINVAL);
  /* Bytes for every length of chunk, and room for the pairs in each. */
  size_t last = 0;
  for (int64_t n = 1; n <= (int64_t)1 << 28; n *= 2) {
    for (int64_t m = n; m <= n + 1 && m <= (int64_t)1 << 28; ++m) {
      const size_t b = dp_embed_grad_workspace(m, (int64_t)1 << 26, 65535 * 64);
      if (b < 16 * (size_t)m || b < last / 2) {
        fprintf(stderr, "FAIL workspace of %lld ids: %zu\n", (long long)m, b);
        ++failures;
      }
      last = b;
    }
  }
}

static void vocabulary(void) {
  float *f = (float*)C, *g = (float*)D;
  int32_t* ti = (int32_t*)W;
  const int64_t big = (int64_t)1 << 31;
  REFUSED(dp_token_logprobs(A, GRZ_BF16, big, 10, 10, B, 64, 0, f, NULL, NULL, NULL, NULL),
          GRZ_ERANGE);
  REFUSED(dp_token_logprobs(A, GRZ_BF16, 4, big, big, B, 64, 0, f, NULL, NULL, NULL, NULL),
          GRZ_ERANGE);
  REFUSED(dp_token_logprobs(A, GRZ_BF16, 4, 10, INT64_MAX, B, 64, 0, f, NULL, NULL, NULL, NULL),
          GRZ_ERANGE);
  REFUSED(dp_token_logprobs(A, GRZ_BF16, 4, 10, 10, B, 64, 11, f, NULL, ti, g, NULL), GRZ_EINVAL);
  REFUSED(dp_token_logprobs(A, GRZ_BF16, 4, 10, 10, B, 64, 2, f, NULL, ti, (float*)A, NULL),
          GRZ_EINVAL);
  REFUSED(dp_token_logprobs(A, GRZ_BF16, 4, 10, 10, B, 64, 2, f, f + 3, ti, g, NULL), GRZ_EINVAL);
  /* the largest row count and width together pass the limit on a matrix's bytes */
  REFUSED(dp_token_logprobs(C, GRZ_F32, big - 1, big - 1, big - 1, B, 64, 0, f, NULL, NULL, NULL,
                            NULL), GRZ_ERANGE);
  /* values over a far element of a large matrix */
  REFUSED(dp_token_logprobs(C, GRZ_F32, (int64_t)1 << 27, big - 1, big - 1, B, 64, 0,
                            (float*)(C + ((int64_t)1 << 58)), NULL, NULL, NULL, NULL), GRZ_EINVAL);
  REFUSED(dp_token_logprobs_grad(A, GRZ_F32, 4, 10, 10, B, 64, NULL, NULL, NULL, NULL, C, 10,
                                 NULL), GRZ_EINVAL);
  REFUSED(dp_token_logprobs_grad(A, GRZ_F32, 4, 10, 10, B, 64, f, NULL, NULL, NULL, B, 10, NULL),
          GRZ_EINVAL);
  REFUSED(dp_token_logprobs_grad(A, GRZ_F32, 4, 10, 10, B, 64, f, NULL, NULL, NULL, A, 12, NULL),
          GRZ_EINVAL);
  REFUSED(dp_distill_loss(A, GRZ_BF16, 4, 10, 10, B, 64, C, GRZ_F32, GRZ_MAX_TOP + 1, 1.0f, NULL,
                          g, NULL), GRZ_EINVAL);
  REFUSED(dp_distill_loss(A, GRZ_BF16, 4, 10, 10, B, 64, C, GRZ_F32, 3, 0.0f, NULL, g, NULL),
          GRZ_EINVAL);
  REFUSED(dp_distill_loss(A, GRZ_BF16, big - 1, 10, 10, B, 64, C, GRZ_F32, 2, 1.0f, NULL, g, NULL),
          GRZ_ERANGE);
  REFUSED(dp_distill_loss(A, GRZ_BF16, 4, 10, 10, B, 64, C, GRZ_F32, 3, 1.0f, NULL, f + 11, NULL),
          GRZ_EINVAL);
  REFUSED(dp_distill_grad(A, GRZ_BF16, 4, 10, 10, B, 64, C, GRZ_F32, 3, 1.0f, NULL, 1.0f, g, D, 10,
                          NULL), GRZ_EINVAL);
  REFUSED(dp_distill_grad(A, GRZ_BF16, 4, 10, 10, B, 64, C, GRZ_F32, 3, 1.0f, NULL, 1.0f, NULL,
                          B + 94, 10, NULL), GRZ_EINVAL);
}

int main(void) {
  embedding();
  vocabulary();
  if (failures) return 1;
  printf("token operators' host checks passed\n");
  return 0;
}
