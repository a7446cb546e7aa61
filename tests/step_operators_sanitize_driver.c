/*
 * Calls the operators around a tree's target pass on every path that a host
 * without a usable GPU reaches -- refused arguments, no-ops, and a device that
 * does not exist -- so that their host side can be built and run under
 * AddressSanitizer and UndefinedBehaviorSanitizer
 * (tests/test_step_operators_sanitized.py).  Every call checks its status code.
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
static void* const FAR = (void*)(uintptr_t)(1 << 30);
enum { NO_DEVICE = 1 << 20 };

static sv_cache cache(void) {
  sv_cache c = {A, A, (float*)A, (float*)A, 0, 4096, 1024, 64, 0, 1, 9, 4, 16, 8, 64};
  return c;
}

static sv_status penalties(const void* logits, void* out, int64_t stride, int V, int B, int nodes, int max_nodes, int cap,
                           const void* mask, int64_t mask_stride) {
  return spec_verify_penalties(logits, SV_BF16, stride, out, SV_BF16, stride, V, A, cap, cap, A, A, A, A, A, B, nodes, max_nodes,
                               A, A, A, A, A, A, 4, mask, mask_stride, 5, NULL, NO_DEVICE, NULL);
}

static sv_status write_rows(const sv_cache* c, const void* k, int64_t row, int B, int nodes, int max_nodes) {
  return spec_verify_cache_write(c, k, A, SV_F32, row, 64, row, 64, A, 3, 3, A, A, B, nodes, max_nodes, NO_DEVICE, NULL);
}

static sv_status keep(const sv_cache* c, const void* path, int depth, int B) {
  return spec_verify_cache_keep(c, path, depth, A, A, 3, 3, A, (int32_t*)FAR, B, NO_DEVICE, NULL);
}

static sv_status attend(const sv_cache* c, const void* q, int64_t q_row, int q_heads, float scale, int B, int nodes,
                        int max_nodes, size_t bytes) {
  return spec_verify_attend(c, q, q_row, 64, FAR, 512, 64, q_heads, scale, A, 3, 3, A, A, A, B, nodes, max_nodes, A, bytes,
                            NO_DEVICE, NULL);
}

int main(void) {
  EXPECT(penalties(A, FAR, 10, 10, 2, 3, 2, 4, A, 1), SV_ECUDA);
  EXPECT(penalties(A, A, 10, 10, 2, 3, 2, 4, A, 1), SV_ECUDA);
  EXPECT(penalties(NULL, NULL, 10, 10, 0, 3, 2, 4, A, 1), SV_OK);
  EXPECT(penalties(A, FAR, 9, 10, 2, 3, 2, 4, A, 1), SV_EINVAL);
  EXPECT(penalties(A, FAR, 100, 100, 2, 3, 2, 4, A, 3), SV_EINVAL);
  EXPECT(penalties(A, FAR, 10, 10, INT32_MIN, 3, 2, 4, A, 1), SV_EINVAL);
  EXPECT(penalties(A, FAR, 10, 10, 2, INT32_MAX, 2, 4, A, 1), SV_EUNSUPPORTED);
  EXPECT(penalties(A, FAR, 10, 10, 2, 3, 2, INT32_MAX, A, 1), SV_EUNSUPPORTED);
  EXPECT(penalties(A, FAR, INT64_MIN, 10, 2, 3, 2, 4, A, 1), SV_EINVAL);

  sv_cache c = cache();
  EXPECT(write_rows(&c, A, 256, 2, 3, 3), SV_ECUDA);
  EXPECT(write_rows(NULL, A, 256, 2, 3, 3), SV_EINVAL);
  EXPECT(write_rows(&c, NULL, 256, 2, 3, 3), SV_EINVAL);
  EXPECT(write_rows(&c, A, INT64_MAX, 2, 3, 3), SV_EUNSUPPORTED);
  EXPECT(write_rows(&c, A, 256, INT32_MAX, 0, INT32_MAX), SV_EUNSUPPORTED);
  EXPECT(write_rows(&c, A, 256, 1 << 28, 1 << 20, INT32_MAX), SV_EUNSUPPORTED);
  EXPECT(keep(&c, A, 2, 2), SV_ECUDA);
  EXPECT(keep(&c, NULL, 2, 2), SV_EINVAL);
  EXPECT(keep(&c, A, INT32_MAX, 2), SV_EUNSUPPORTED);
  EXPECT(keep(&c, A, 2, INT32_MAX), SV_EUNSUPPORTED);
  c.layers = INT32_MAX, c.layer_stride = (int64_t)1 << 39;
  EXPECT(keep(&c, A, 2, INT32_MAX), SV_EUNSUPPORTED);
  EXPECT(write_rows(&c, A, 256, 2, 3, 3), SV_EINVAL);
  c = cache();
  c.page_stride = INT64_MIN;
  EXPECT(keep(&c, A, 2, 2), SV_EINVAL);
  c = cache();
  c.block = INT32_MIN;
  EXPECT(keep(&c, A, 2, 2), SV_EINVAL);

  c = cache();
  EXPECT(attend(&c, A, 512, 8, 0.1f, 2, 3, 3, SIZE_MAX), SV_ECUDA);
  EXPECT(attend(&c, A, 512, 8, 0.1f, 0, 3, 3, 0), SV_OK);
  EXPECT(attend(&c, A, 512, 6, 0.1f, 2, 3, 3, SIZE_MAX), SV_EINVAL);
  EXPECT(attend(&c, A, 512, 8, NAN, 2, 3, 3, SIZE_MAX), SV_EINVAL);
  EXPECT(attend(&c, A, INT64_MIN, 8, 0.1f, 2, 3, 3, SIZE_MAX), SV_EINVAL);
  EXPECT(attend(&c, A, 512, 8, 0.1f, 2, 3, INT32_MAX, SIZE_MAX), SV_EUNSUPPORTED);
  EXPECT(attend(&c, A, 512, INT32_MAX - 3, 0.1f, 2, 3, 3, SIZE_MAX), SV_EUNSUPPORTED);
  if (spec_verify_attend_workspace(4, 8, 64, 3, NO_DEVICE) != 0 || spec_verify_attend_workspace(0, 8, 64, 3, 0) != 0) ++failures;

  printf("%d failed checks\n", failures);
  return failures != 0;
}
