/*
 * Host-side checks of the mixture-of-experts operators and of the lists of tensors,
 * built and run by tests/test_experts_native.py against the regular library and
 * against their sources with AddressSanitizer in their host code.  Only host logic
 * runs: sizes, and argument errors that are reported before anything is enqueued (no
 * call here reaches a kernel launch; the device pointers passed are never
 * dereferenced).
 */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "grz.h"

#ifdef WITHOUT_STEP
/* The norm's tree is the step's, whose source is not in the instrumented library: its
 * size for the few pieces below, and no call that reaches its launch. */
size_t dp_grad_sqnorm_workspace(int64_t npieces) { return npieces <= 4096 ? 0 : (size_t)-1; }
int dp_grad_sqnorm(const double* piece_sqnorm, int64_t npieces, double max_norm, void* workspace,
                   double* sqnorm_out, float* clip_scale_out, hipStream_t stream) {
  (void)piece_sqnorm, (void)npieces, (void)max_norm, (void)workspace;
  (void)sqnorm_out, (void)clip_scale_out, (void)stream;
  return GRZ_EHIP;
}
#endif

static int failures = 0;
#define REFUSED(call, want)                                                         \
  do {                                                                              \
    const long long got = (long long)(call);                                        \
    if (got != (long long)(want)) {                                                 \
      fprintf(stderr, "FAIL %s:%d: %s: %lld\n", __FILE__, __LINE__, #call, got);    \
      ++failures;                                                                   \
    }                                                                               \
  } while (0)

static char* const A = (char*)0x100000;
static char* const B = (char*)0x20000000;
static char* const C = (char*)0x40000000;
static char* const D = (char*)0x60000000;
static char* const E = (char*)0x80000000;

static void experts(void) {
  int32_t* const ids = (int32_t*)B;
  int32_t* const places = (int32_t*)C;
  float* const w = (float*)D;
  const int64_t limits[] = {INT64_MIN, -1, (int64_t)1 << 31, (int64_t)1 << 62, INT64_MAX};
  for (int i = 0; i < 5; ++i) {
    const int64_t v = limits[i];
    const int want = v < 0 ? GRZ_EINVAL : GRZ_ERANGE;
    REFUSED(dp_expert_route(A, GRZ_BF16, v, 8, 8, 2, 0, ids, w, NULL), want);
    REFUSED(dp_expert_route(A, GRZ_BF16, 4, v, v, 1, 0, ids, w, NULL), want);
    REFUSED(dp_expert_route_grad(A, GRZ_F32, v, 8, 8, 2, 0, ids, w, E, 8, NULL), want);
    REFUSED(dp_expert_sort(A, 64, v, 2, 8, E, ids, places, NULL), want);
    REFUSED(dp_expert_sort(A, 64, 4, 2, v, E, ids, places, NULL), want);
    REFUSED(dp_expert_sort_workspace(v, 2, 8), 0);
    REFUSED(dp_expert_sort_workspace(1 << 20, 2, v), 0);
    REFUSED(dp_expert_dispatch(A, GRZ_BF16, 8, places, w, v, 2, 8, 8, E, GRZ_BF16, 8, NULL), want);
    REFUSED(dp_expert_dispatch(A, GRZ_BF16, v, places, w, 4, 2, v, 8, E, GRZ_BF16, v, NULL), want);
    REFUSED(dp_expert_dispatch(A, GRZ_BF16, 8, places, w, 4, 2, 8, v, E, GRZ_BF16, 8, NULL), want);
    REFUSED(dp_expert_combine(A, GRZ_F32, 8, v, places, w, 4, 2, 8, 0, E, GRZ_F32, 8, NULL), want);
    REFUSED(dp_expert_combine(A, GRZ_F32, 8, 8, places, w, v, 2, 8, 0, E, GRZ_F32, 8, NULL), want);
    REFUSED(dp_expert_combine_grad(A, GRZ_F32, 8, B, GRZ_F32, 8, v, places, w, 4, 2, 8, E, 8, NULL,
                                   NULL), want);
    REFUSED(dp_expert_combine_grad(A, GRZ_F32, 8, B, GRZ_F32, 8, 8, places, w, v, 2, 8, E, 8, NULL,
                                   NULL), want);
  }
  REFUSED(dp_expert_dispatch(A, GRZ_BF16, INT64_MAX, places, w, 4, 2, 8, 8, E, GRZ_BF16, 8, NULL),
          GRZ_ERANGE);
  REFUSED(dp_expert_route(A, GRZ_BF16, 4, 8, 8, INT32_MAX, 0, ids, w, NULL), GRZ_EINVAL);
  REFUSED(dp_expert_route(A, GRZ_BF16, 4, 8, 8, INT32_MIN, 0, ids, w, NULL), GRZ_EINVAL);
  for (int64_t m = 1; m <= (int64_t)1 << 28; m *= 2)
    if (dp_expert_sort_workspace(m, 1, GRZ_MAX_EXPERTS) > (size_t)1 << 20) {
      fprintf(stderr, "FAIL workspace of %lld slots\n", (long long)m);
      ++failures;
    }
}

/* Lists of every length around what one launch and the stack hold. */
static void lists(void) {
  for (int64_t n = 0; n <= 400; n += n < 40 ? 1 : 9) {
    grz_tensor* t = (grz_tensor*)malloc((size_t)(n + 1) * sizeof *t);
    grz_tensor* o = (grz_tensor*)malloc((size_t)(n + 1) * sizeof *o);
    for (int64_t i = 0; i < n; ++i) {
      /* in a scattered order of addresses */
      const int64_t at = (i * 7) % (n > 0 && n % 7 == 0 ? n + 1 : n);
      t[i].data = A + at * 4096;
      t[i].numel = 1000;
      t[i].dtype = i % 2 ? GRZ_BF16 : GRZ_F32;
      o[i] = t[i];
      o[i].data = B + at * 4096;
    }
    REFUSED(dp_tensor_pieces(t, n), n);
    REFUSED(dp_grad_sqnorm_tensors_workspace(t, n, 3), 8 * (size_t)(n + 3));
    if (n > 1) {
      o[n - 1].data = o[0].data; /* two outputs in one place */
      REFUSED(dp_grad_clip_tensors(t, n, (float*)E, o, NULL), GRZ_EINVAL);
      o[n - 1].data = t[0].data; /* another gradient's place */
      REFUSED(dp_grad_clip_tensors(t, n, (float*)E, o, NULL), GRZ_EINVAL);
      t[n - 1].data = (char*)t[0].data + 996;
      REFUSED(dp_grad_clip_tensors(t, n, (float*)E, NULL, NULL), GRZ_EINVAL);
      REFUSED(dp_grad_sqnorm_tensors(t, n, 1.0, 0, t[0].data, (double*)D, NULL, NULL), GRZ_EINVAL);
    }
    if (n > 0) {
      t[n - 1].numel = INT64_MAX;
      REFUSED(dp_tensor_pieces(t, n), -GRZ_ERANGE);
      REFUSED(dp_grad_clip_tensors(t, n, NULL, NULL, NULL), GRZ_ERANGE);
      t[n - 1].numel = INT64_MIN;
      REFUSED(dp_tensor_pieces(t, n), -GRZ_EINVAL);
      REFUSED(dp_grad_sqnorm_tensors(t, n, 1.0, 0, C, (double*)D, NULL, NULL), GRZ_EINVAL);
    }
    free(t);
    free(o);
  }
  REFUSED(dp_tensor_pieces(NULL, 1), -GRZ_EINVAL);
  REFUSED(dp_tensor_pieces(NULL, -1), -GRZ_EINVAL);
  REFUSED(dp_grad_clip_tensors(NULL, INT64_MIN, NULL, NULL, NULL), GRZ_EINVAL);
}

int main(void) {
  experts();
  lists();
  if (failures) return 1;
  printf("experts' host checks passed\n");
  return 0;
}
