/*
 * Calls the operators around a verifying call on every path that a host
 * without a usable GPU reaches -- refused arguments, no-ops, and a device that
 * does not exist -- so that their host side can be built and run under
 * AddressSanitizer and UndefinedBehaviorSanitizer
 * (tests/test_operators_sanitized.py).  Every call checks its status code.
 */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "spec_verify.h"

static int failures = 0;
#define EXPECT(call, want)                                                                 \
  do {                                                                                     \
    const sv_status got_ = (call);                                                         \
    if (got_ != (want)) {                                                                  \
      fprintf(stderr, "%s:%d: returned %d, expected %d\n", __FILE__, __LINE__, (int)got_, (int)(want)); \
      ++failures;                                                                          \
    }                                                                                      \
  } while (0)

/* never read: every call is refused, does nothing, or names a device that does not exist */
static void* const A = (void*)(uintptr_t)(1 << 20);
enum { NO_DEVICE = 1 << 20 };

static sv_status linear(const void* x, const void* w, void* y, int64_t x_row, int64_t y_row, int64_t y_group, int groups,
                        int M, int N, int K, sv_activation act, float cap) {
  return spec_verify_linear(x, x_row, 0, w, 64, 0, NULL, SV_F32, 0, NULL, SV_F32, 0, 0, y, SV_BF16, y_row, y_group, groups,
                            M, N, K, act, cap, NO_DEVICE, NULL);
}

static sv_status softmax(const void* logits, void* probs, int64_t stride, int rows, int V, float t) {
  return spec_verify_softmax(logits, SV_BF16, stride, rows, V, t, NULL, (float*)probs, stride, NO_DEVICE, NULL);
}

static sv_status tree(const void* p, const void* q, int B, int nodes, int max_nodes, int max_depth, int V, void* tokens) {
  return spec_verify_tree((const float*)p, V, (const float*)q, V, 2, A, A, A, A, A, A, B, nodes, max_nodes, max_depth, V,
                          SV_WITH_REPLACEMENT, tokens, tokens, NULL, NULL, NULL, NULL, NO_DEVICE, NULL);
}

int main(void) {
  EXPECT(linear(A, A, A, 64, 32, 128, 2, 4, 32, 64, SV_ACT_NONE, 0.f), SV_ECUDA);
  EXPECT(linear(A, A, A, 64, 32, 128, 0, 4, 32, 64, SV_ACT_NONE, 0.f), SV_OK);
  EXPECT(linear(A, A, A, 64, 32, 128, 2, -4, 32, 64, SV_ACT_NONE, 0.f), SV_EINVAL);
  EXPECT(linear(NULL, A, A, 64, 32, 128, 2, 4, 32, 64, SV_ACT_NONE, 0.f), SV_EINVAL);
  EXPECT(linear(A, A, NULL, 64, 32, 128, 2, 4, 32, 64, SV_ACT_NONE, 0.f), SV_EINVAL);
  EXPECT(linear(A, A, A, 64, 31, 128, 2, 4, 32, 64, SV_ACT_NONE, 0.f), SV_EINVAL);
  EXPECT(linear(A, A, A, 64, INT64_MAX, INT64_MAX, 2, 4, 32, 64, SV_ACT_NONE, 0.f), SV_EUNSUPPORTED);
  EXPECT(linear(A, A, A, INT64_MIN, 32, 128, 2, 4, 32, 64, SV_ACT_NONE, 0.f), SV_EINVAL);
  EXPECT(linear(A, A, A, 64, 32, 128, 2, 4, 32, INT32_MAX, SV_ACT_NONE, 0.f), SV_EUNSUPPORTED);
  EXPECT(linear(A, A, A, 64, (int64_t)1 << 39, (int64_t)1 << 31, 1 << 30, 1 << 30, 1 << 30, 64, SV_ACT_NONE, 0.f),
         SV_EINVAL);
  EXPECT(linear(A, A, A, 64, (int64_t)1 << 39, ((int64_t)1 << 39) + 1, 1 << 30, 1 << 30, 1, 64, SV_ACT_NONE, 0.f),
         SV_EINVAL);
  EXPECT(linear(A, A, A, 64, 32, 128, 2, 4, 32, 64, (sv_activation)6, 0.f), SV_EINVAL);
  EXPECT(linear(A, A, A, 64, 32, 128, 2, 4, 32, 64, SV_ACT_SOFTCAP, NAN), SV_EINVAL);

  EXPECT(softmax(A, A, 10, 2, 10, 1.f), SV_ECUDA);
  EXPECT(softmax(NULL, NULL, 10, 0, 10, 1.f), SV_OK);
  EXPECT(softmax(A, NULL, 10, 2, 10, 1.f), SV_EINVAL);
  EXPECT(softmax(A, A, 9, 2, 10, 1.f), SV_EINVAL);
  EXPECT(softmax(A, A, 10, 2, 10, INFINITY), SV_EINVAL);
  EXPECT(softmax(A, A, (int64_t)1 << 40, 2, SV_MAX_V + 1, 1.f), SV_EUNSUPPORTED);
  EXPECT(softmax(A, A, 10, INT32_MIN, 10, 1.f), SV_EINVAL);

  EXPECT(tree(A, A, 2, 3, 2, 2, 10, A), SV_ECUDA);
  EXPECT(tree(NULL, NULL, 0, 0, 0, 0, 10, NULL), SV_OK);
  EXPECT(tree(NULL, A, 2, 3, 2, 2, 10, A), SV_EINVAL);
  EXPECT(tree(A, A, 2, 3, 2, 2, 10, NULL), SV_EINVAL);
  EXPECT(tree(A, A, 2, 3, SV_MAX_NODES + 1, 2, 10, A), SV_EUNSUPPORTED);
  EXPECT(tree(A, A, INT32_MIN, 3, 2, 2, 10, A), SV_EINVAL);
  EXPECT(tree(A, A, 2, 3, 2, INT32_MAX, 10, A), SV_EINVAL);

  printf("%d failed checks\n", failures);
  return failures != 0;
}
