/* Argument checks of the row operators, driven from C without a GPU: every call here is
 * refused, or has nothing to do, before anything is enqueued. */
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "w4a16_moe.h"

static int failures = 0;
#define EXPECT(status, call)                                                               \
  do {                                                                                     \
    const int rc_ = (call);                                                                \
    if (rc_ != (status)) {                                                                 \
      ++failures;                                                                          \
      printf("line %d: %d, expected %d (%s)\n", __LINE__, rc_, (status), moe_last_error()); \
    }                                                                                      \
  } while (0)

static const int sizes[] = {INT_MIN, -1, 0, 1, 7, 8, 1024, 1 << 20, 1 << 24, (1 << 24) + 1, INT_MAX};
#define NUM_SIZES ((int)(sizeof(sizes) / sizeof(sizes[0])))

int main(void) {
  /* never dereferenced: a valid address for the alignment checks only */
  void* p = aligned_alloc(256, 256);
  float* f = (float*)p;
  int32_t* pos = (int32_t*)p;
  int calls = 0;
  /* sizes of every kind with a missing pointer: refused whatever the sizes are, or no tokens */
  for (int i = 0; i < NUM_SIZES; ++i)
    for (int j = 0; j < NUM_SIZES; ++j)
      for (int k = 0; k < NUM_SIZES; ++k) {
        const int T = sizes[i], d = sizes[j], n = sizes[k];
        const int a = moe_permute(NULL, d, MOE_BF16, T, d, n, pos, f, p, d, n, NULL);
        const int b = moe_unpermute(p, d, n, MOE_FP16, T, d, n, pos, f, NULL, d, NULL);
        const int c = moe_permute_backward(p, d, n, p, d, MOE_FP32, T, d, n, pos, f, NULL, d, f, NULL);
        const int e = moe_unpermute_backward(NULL, d, p, d, MOE_BF16, T, d, n, pos, f, p, d, n, f, NULL);
        if (T > 0 && (a == MOE_OK || b == MOE_OK || c == MOE_OK || e == MOE_OK)) {
          ++failures;
          printf("accepted T=%d d=%d n=%d\n", T, d, n);
        }
        moe_route_backward_args r;
        memset(&r, 0, sizeof(r));
        r.T = T;
        r.d = d;
        r.E = n;
        r.k = 1;
        r.renormalize = 1;
        if (moe_route_backward(&r, NULL) == MOE_OK && T != 0) {
          ++failures;
          printf("route_backward accepted T=%d d=%d E=%d\n", T, d, n);
        }
        moe_block_norm_args b_args;
        memset(&b_args, 0, sizeof(b_args));
        b_args.T = T;
        b_args.d = d;
        b_args.x_stride = n;
        b_args.eps = 1e-6f;
        moe_block_norm_grads g;
        memset(&g, 0, sizeof(g));
        if ((moe_block_norm(&b_args, NULL, n, NULL, n, NULL) == MOE_OK ||
             moe_block_norm_backward(&b_args, &g, NULL) == MOE_OK) &&
            T != 0) {
          ++failures;
          printf("block_norm accepted T=%d d=%d\n", T, d);
        }
        const int64_t w = moe_route_backward_workspace_bytes(T, d, n, 8);
        const int64_t v = moe_block_norm_backward_workspace_bytes(T, d);
        if ((T < 0 || d <= 0 || n <= 0) ? w != -1 : w == 0 || w < -1) ++failures;
        if ((T < 0 || d <= 0) ? v != -1 : v < 0) ++failures;
        calls += 9;
      }
  EXPECT(MOE_ERR_INVALID_ARG, moe_route_backward(NULL, NULL));
  EXPECT(MOE_ERR_INVALID_ARG, moe_block_norm(NULL, p, 8, p, 8, NULL));
  EXPECT(MOE_ERR_INVALID_ARG, moe_block_norm_backward(NULL, NULL, NULL));
  moe_block_norm_args a;
  memset(&a, 0, sizeof(a));
  a.T = 2;
  a.d = 8;
  a.x = a.y = a.norm_out = a.norm_in = p;
  a.x_stride = a.y_stride = 8;
  const float bad[] = {0.f, -1.f, 1e-40f, NAN, INFINITY};
  for (int i = 0; i < 5; ++i) {
    a.eps = bad[i];
    EXPECT(MOE_ERR_INVALID_ARG, moe_block_norm(&a, p, 8, p, 8, NULL));
  }
  a.eps = 1e-6f;
  for (int kind = -1; kind <= 4; ++kind) {
    a.gate_kind = kind;
    if (kind != MOE_GATE_NONE) EXPECT(MOE_ERR_INVALID_ARG, moe_block_norm(&a, p, 8, p, 8, NULL));
  }
  free(p);
  printf("row checks: %d calls, %d failures\n", calls, failures);
  return failures != 0;
}
